"""Cases of the paged shared cache's operators, their plain forms and their exact values.

Four operators make one decode step over a paged cache: ``plan`` (block tables and slot
maps from request lengths), ``append`` (new tokens' rows into their pages, with each page's
key bounds), ``decode`` (attention of one new token per sequence over the pages) and
``sparse`` (the same over the pages that a cheap score selects for each kv head).

``own`` chooses between the plain forms (elementary torch operations in 32 bits) and the
calls a user makes of the framework. ``exact`` is the definition in 64 bits, written apart.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the step of a running batch: every request takes one more token
        dict(name="plan_step", op="plan", batch=64, page=64, max_blocks=64, tokens=64, kind="step", lens_seed=1),
        # continuous batching: prompts arrive in chunks beside running requests, finished ones leave
        dict(name="plan_mixed", op="plan", batch=509, page=16, max_blocks=1024, tokens=65536, kind="mixed", lens_seed=2),
        # one token of each of 32 requests (1.1B CLA2 head layout), bounds not kept
        dict(name="append_step", op="append", dtype="bf16", batch=32, kv_heads=4, q_heads=32, d=64, page=64,
             max_blocks=32, tokens=32, bounds=False, lens_seed=3),
        # prompt chunks of a few requests, K and V read in place from the fused projection's rows, bounds kept
        dict(name="append_prompts", op="append", dtype="bf16", batch=7, kv_heads=8, q_heads=32, d=128, page=64,
             max_blocks=64, tokens=8191, bounds=True, lens_seed=4),
        # fp32 cache, small odd chunk
        dict(name="append_f32", op="append", dtype="f32", batch=5, kv_heads=2, q_heads=4, d=64, page=16,
             max_blocks=40, tokens=333, bounds=False, lens_seed=5),
        # one request with a short context: latency
        dict(name="decode_one", op="decode", dtype="bf16", batch=1, kv_heads=4, q_heads=16, d=128, page=16,
             max_blocks=20, mix=False, lens_seed=6),
        # a batch of ragged requests on the 1.1B CLA2 layout
        dict(name="decode_batch", op="decode", dtype="bf16", batch=32, kv_heads=4, q_heads=32, d=64, page=64,
             max_blocks=32, mix=False, lens_seed=7),
        # a target layer that mixes two source layers, 8K contexts
        dict(name="decode_mix", op="decode", dtype="bf16", batch=16, kv_heads=4, q_heads=16, d=128, page=32,
             max_blocks=256, mix=True, lens_seed=8),
        # long contexts: a few requests of up to 64K tokens
        dict(name="decode_long", op="decode", dtype="bf16", batch=4, kv_heads=8, q_heads=32, d=128, page=128,
             max_blocks=512, mix=False, lens_seed=9),
        # fp32 cache
        dict(name="decode_f32", op="decode", dtype="f32", batch=9, kv_heads=2, q_heads=8, d=64, page=16,
             max_blocks=128, mix=False, lens_seed=10),
        # one request, 32 of its pages
        dict(name="sparse_one", op="sparse", dtype="bf16", batch=1, kv_heads=8, q_heads=32, d=128, page=32,
             max_blocks=512, top=32, mix=False, lens_seed=11),
        # long contexts, 64 of up to 1024 pages per kv head
        dict(name="sparse_long", op="sparse", dtype="bf16", batch=8, kv_heads=8, q_heads=32, d=128, page=64,
             max_blocks=1024, top=64, mix=False, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "sparse"])
    seed = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        tokens = _log(rng, 16, 65536)
        return dict(op=op, batch=_log(rng, 1, 509), page=page, max_blocks=_log(rng, 8, 1024), tokens=tokens,
                    kind=rng.choice(["step", "mixed"]), lens_seed=seed)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 8, 16])
    c = dict(op=op, dtype=dtype, kv_heads=kv_heads, q_heads=kv_heads * g, d=d, page=page, lens_seed=seed)
    if op == "append":
        tokens = _log(rng, 1, 8191)
        c.update(batch=_log(rng, 1, 64), tokens=tokens, bounds=rng.random() < 0.5)
        c["max_blocks"] = -(-(2 * tokens // c["batch"] + 600) // page)
        return c
    # a decode or sparse step reads at most about what the largest listed one does
    batch = _log(rng, 1, 64)
    most = 4 * 65536 * 8 * 128 * 2 // (batch * kv_heads * d * (2 if dtype == "bf16" else 4))
    c.update(batch=batch, mix=rng.random() < 0.3)
    c["max_blocks"] = max(2, _log(rng, 40, max(64, min(65536, most // (2 if c["mix"] else 1)))) // page)
    if op == "sparse":
        c["top"] = max(3, min(c["max_blocks"], _log(rng, 4, 128)))
    return c


def _lengths(case):
    """Tokens of each sequence: ragged, the first one full, every eighth row of a batch idle."""
    r = random.Random(case["lens_seed"])
    cap = case["max_blocks"] * case["page"]
    lens = [max(1, int(cap * r.uniform(0.3, 1.0))) for _ in range(case["batch"])]
    lens[0] = cap - r.randrange(0, case["page"])
    for b in range(7, case["batch"], 8):
        lens[b] = 0
    return lens


def _new_tokens(case):
    """(cached tokens, new tokens) of each sequence for an append or a plan."""
    r = random.Random(case["lens_seed"])
    B, cap, total = case["batch"], case["max_blocks"] * case["page"], case["tokens"]
    if case["op"] == "append":
        cuts = sorted(r.randrange(0, total + 1) for _ in range(B - 1))
        new = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        if total == B:
            new = [1] * B
        new = [min(n, cap) for n in new]
        return [r.randrange(0, cap - n + 1) for n in new], new
    old = [r.randrange(0, cap) for _ in range(B)]
    if case["kind"] == "step":
        return old, [1 if i < total else 0 for i in range(B)]
    new = [1] * B
    for b in range(B):
        x = r.random()
        if x < 0.1:
            new[b] = -1                                          # finished: its pages return
        elif x < 0.3:
            old[b] = 0
            new[b] = r.randrange(1, max(2, min(cap, 8 * total // B)))   # a prompt chunk
    return old, new


# ------------------------------------------------------------------------------ inputs
def _mix_weights(kv_heads):
    """A target layer's weight of its first source, per kv head: fixed by the model, not by the request."""
    return [0.25 + 0.5 * (j + 1) / (kv_heads + 1) for j in range(kv_heads)]


def _bounds_of(k, rows):
    """Bounds of the first `rows` [...] keys of pages k [..., page, d]: int8 codes [..., 2, d] and scales."""
    keep = torch.arange(k.shape[-2], device=k.device) < rows[..., None]
    x = k.float()
    hi = x.masked_fill(~keep[..., None], -math.inf).amax(-2)
    lo = x.masked_fill(~keep[..., None], math.inf).amin(-2)
    some = (rows > 0)[..., None]
    hi, lo = hi.where(some, 0.0), lo.where(some, 0.0)
    scale = torch.maximum(hi.abs(), lo.abs()).amax(-1) / 127.0
    safe = scale.where(scale > 0, 1.0)[..., None]
    ch = torch.ceil(hi / safe).clamp(max=127.0)
    cl = torch.floor(lo / safe).clamp(min=-127.0)
    codes = torch.stack([ch, cl], -2) * (scale > 0)[..., None, None]
    return codes.to(torch.int8), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, ps, P = case["batch"], case["page"], case["max_blocks"]
    s = dict(case=case)
    ints = dict(dtype=torch.int32, device=dev)
    if case["op"] == "plan":
        old, new = _new_tokens(case)
        held = [-(-n // ps) for n in old]
        wanted = sum(max(0, -(-(n + max(m, 0)) // ps) - h) for n, m, h in zip(old, new, held))
        s["num_pages"] = N = sum(held) + wanted + 37
        ids = torch.randperm(N, generator=gen, device=dev).to(torch.int32)
        table = torch.full((B, P), -1, **ints)
        col = torch.arange(P, device=dev)
        held_t = torch.tensor(held, device=dev)
        first = held_t.cumsum(0) - held_t
        used = col < held_t[:, None]
        table = torch.where(used, ids[(first[:, None] + col).clamp(max=N - 1)], table)
        ring = torch.full((N,), -1, **ints)
        head = int(seed) % N
        free = ids[sum(held):]
        ring[(head + torch.arange(len(free), device=dev)) % N] = free
        s.update(block_table=table, ring=ring, ring_state=torch.tensor([head, len(free)], **ints),
                 lengths=torch.tensor(old, **ints), new_tokens=torch.tensor(new, **ints),
                 lengths_out=torch.zeros(B, **ints), ring_state_out=torch.zeros(2, **ints),
                 token_start=torch.zeros(B + 1, **ints), slot_map=torch.zeros(case["tokens"], **ints),
                 position=torch.zeros(case["tokens"], **ints))
        return s
    dt, Hkv, Hq, d = DTYPES[case["dtype"]], case["kv_heads"], case["q_heads"], case["d"]
    slots = 2 if case.get("mix") else 1
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=dev).to(dt)  # noqa: E731
    N = B * P + 3
    s["block_table"] = (torch.randperm(N, generator=gen, device=dev)[: B * P].to(torch.int32)).view(B, P)
    s["k"], s["v"] = rand(slots, N, Hkv, ps, d), rand(slots, N, Hkv, ps, d)
    if case["op"] == "append":
        old, new = _new_tokens(case)
        rows = torch.cat([torch.arange(n, n + m, device=dev) for n, m in zip(old, new)])
        seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(new, device=dev))
        slot = s["block_table"][seq, rows // ps].long() * ps + rows % ps
        pad = case["tokens"] - len(rows)
        s["slot_map"] = torch.cat([slot, torch.full((pad,), -1, device=dev)]).to(torch.int32)
        qkv = rand(case["tokens"], Hq + 2 * Hkv, d)             # the fused projection's rows
        s["k_new"], s["v_new"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["lengths"] = torch.tensor([n + m for n, m in zip(old, new)], **ints)
        if case["bounds"]:
            s["bound_codes"] = torch.zeros(slots, N, Hkv, 2, d, dtype=torch.int8, device=dev)
            s["bound_scale"] = torch.zeros(slots, N, Hkv, device=dev)
        return s
    s["q"] = rand(1, B, Hq, d) * 2                              # [layers][B][Hq][d], one layer
    s["lengths"] = torch.tensor(_lengths(case), **ints)
    s["out"] = torch.empty(1, B, Hq, d, device=dev)
    s["lse"] = torch.empty(1, B, Hq, device=dev)
    if case["op"] == "sparse":
        # keys of a page lie around a direction of their own, as neighbouring tokens' do
        s["k"] += (1.5 * torch.randn(slots, N, Hkv, 1, d, generator=gen, device=dev)).to(dt)
        held = torch.zeros(N, dtype=torch.int64, device=dev)
        here = (s["lengths"][:, None] - torch.arange(P, device=dev) * ps).clamp(0, ps)
        held[s["block_table"].long()] = here.long()
        s["bound_codes"], s["bound_scale"] = _bounds_of(s["k"], held[None, :, None].expand(slots, N, Hkv))
        s["selected"] = torch.empty(1, B, Hkv, case["top"], **ints)
    return s


# ------------------------------------------------------------------------- plain forms
def _plain_plan(s):
    c = s["case"]
    ps, B, P, N, M = c["page"], c["batch"], c["max_blocks"], s["num_pages"], c["tokens"]
    n, m = s["lengths"].long(), s["new_tokens"].long()
    head, count = s["ring_state"].long()
    dev = n.device
    held = (n + ps - 1) // ps
    leaving = m < 0
    want = m.clamp(min=0)
    want = want * (n + want <= P * ps)
    need = (n + want + ps - 1) // ps - held
    fits = ((need.cumsum(0) <= count) | (need == 0)) & (want.cumsum(0) <= M)
    got, need = want * fits, need * fits
    back = held * leaving
    kept = back.cumsum(0) <= N - count
    back = back * kept
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), got.cumsum(0)])
    col = torch.arange(P, device=dev)
    # new pages: the k-th one of the call is the ring's k-th from its head
    k = (need.cumsum(0) - need)[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, s["ring"].long()[(head + k) % N], s["block_table"].long())
    # pages of sequences that leave go behind the ring's last
    r = (back.cumsum(0) - back)[:, None] + col
    at = torch.where(col < back[:, None], (head + count + r) % N, N)
    ring = torch.cat([s["ring"].long(), torch.zeros(1, dtype=torch.int64, device=dev)])
    ring = ring.scatter(0, at.reshape(-1), s["block_table"].long().reshape(-1))[:N]
    i = torch.arange(M, device=dev)
    b = torch.searchsorted(start[1:], i, right=True).clamp(max=B - 1)
    live = i < start[-1]
    pos = torch.where(live, n[b] + i - start[b], 0)
    slot = torch.where(live, table[b, (pos // ps).clamp(max=P - 1)] * ps + pos % ps, -1)
    state = torch.stack([(head + need.sum()) % N, count - need.sum() + back.sum()])
    as_int = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(block_table=as_int(table), ring=as_int(ring), ring_state=as_int(state), token_start=as_int(start),
                lengths=as_int(torch.where(leaving, 0, n + got)), slot_map=as_int(slot), position=as_int(pos))


def _plain_append(s):
    c = s["case"]
    ps = c["page"]
    slot = s["slot_map"].long()
    live = slot >= 0
    page, row = slot[live] // ps, slot[live] % ps
    k, v = s["k"], s["v"]
    k[0].transpose(1, 2)[page, row] = s["k_new"][live]
    v[0].transpose(1, 2)[page, row] = s["v_new"][live]
    if not c["bounds"]:
        return dict(k=k, v=v)
    # a page's bounds cover its rows up to the last one written here
    last = torch.zeros(k.shape[1], dtype=torch.int64, device=k.device).scatter_reduce(0, page, row + 1, "amax")
    touched = last > 0
    codes, scale = _bounds_of(k[0], last[:, None].expand(-1, c["kv_heads"]))
    s["bound_codes"][0] = codes.where(touched[:, None, None, None], s["bound_codes"][0])
    s["bound_scale"][0] = scale.where(touched[:, None], s["bound_scale"][0])
    return dict(k=k, v=v, bounds=s["bound_codes"].float() * s["bound_scale"][..., None, None])


def _attend(c, q, keys, values, valid, w):
    """q [B,Hkv,g,d] over per-source keys and values [B,Hkv,n,d]; valid [B,1 or Hkv,n]."""
    if len(keys) == 1:
        k, v = keys[0].float(), values[0].float()
    else:
        x = w[:, None, None]
        k = x * keys[0].float() + (1.0 - x) * keys[1].float()
        v = x * values[0].float() + (1.0 - x) * values[1].float()
    scores = (q @ k.transpose(-1, -2)) / math.sqrt(c["d"])
    scores = scores.masked_fill(~valid[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = top.where(top > -math.inf, 0.0)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.where(total > 0, 1.0)
    lse = (top + torch.log(total))[..., 0]
    B, Hkv, g, d = q.shape
    return out.reshape(1, B, Hkv * g, d), lse.reshape(1, B, Hkv * g)


def _sources(c):
    return (0, 1) if c["mix"] else (0,)


def _weights(c, device):
    return torch.tensor(_mix_weights(c["kv_heads"]), dtype=torch.float32, device=device)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, d, ps, P = c["batch"], c["kv_heads"], c["d"], c["page"], c["max_blocks"]
    table = s["block_table"].long()
    pages = lambda pool, src: pool[src][table].transpose(1, 2).reshape(B, Hkv, P * ps, d)  # noqa: E731
    valid = torch.arange(P * ps, device=table.device) < s["lengths"][:, None]
    q = s["q"][0].float().view(B, Hkv, -1, d)
    out, lse = _attend(c, q, [pages(s["k"], x) for x in _sources(c)], [pages(s["v"], x) for x in _sources(c)],
                       valid[:, None], _weights(c, table.device))
    return dict(out=out, lse=lse)


def _plain_select(s):
    """The block indices [B,Hkv,top] each kv head keeps: its first page, its last, then the highest scores."""
    c = s["case"]
    B, Hkv, d, ps, P, K = c["batch"], c["kv_heads"], c["d"], c["page"], c["max_blocks"], c["top"]
    table = s["block_table"].long()
    q = s["q"][0].float().view(B, Hkv, -1, d)
    sq = q.abs().amax(-1, keepdim=True) / 127.0
    qc = torch.round(q / sq.where(sq > 0, 1.0)) * (sq > 0)
    scores = []
    for src in _sources(c):                                      # one or two source layers
        codes = s["bound_codes"][src][table].transpose(1, 2).float()          # [B,Hkv,P,2,d]
        # whole numbers below 2^24: exact in 32 bits whatever the order
        dot = qc.clamp(min=0) @ codes[..., 0, :].transpose(-1, -2) + qc.clamp(max=0) @ codes[..., 1, :].transpose(-1, -2)
        scale = s["bound_scale"][src][table].transpose(1, 2)
        scores.append(dot * sq * scale[:, :, None])
    if c["mix"]:
        w = _weights(c, table.device)[:, None, None]
        score = w * scores[0] + (1.0 - w) * scores[1]
    else:
        score = scores[0]
    score = score.amax(2)                                        # [B,Hkv,P]
    held = ((s["lengths"].long() + ps - 1) // ps)[:, None, None]
    col = torch.arange(P, device=table.device)
    score = score.masked_fill((col == 0) | (col == held - 1), math.inf).masked_fill(col >= held, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :K]
    order = order.masked_fill((order >= held), P).sort(-1).values
    return order.masked_fill(order == P, -1)


def _plain_sparse(s):
    c = s["case"]
    B, Hkv, d, ps, K = c["batch"], c["kv_heads"], c["d"], c["page"], c["top"]
    chosen = _plain_select(s)
    pick = torch.gather(s["block_table"].long()[:, None].expand(B, Hkv, -1), 2, chosen.clamp(min=0))
    j = torch.arange(Hkv, device=pick.device)[None, :, None]
    pages = lambda pool, src: pool[src][pick, j].reshape(B, Hkv, K * ps, d)  # noqa: E731
    at = chosen[..., None] * ps + torch.arange(ps, device=pick.device)
    valid = ((chosen >= 0)[..., None] & (at < s["lengths"][:, None, None, None])).reshape(B, Hkv, K * ps)
    q = s["q"][0].float().view(B, Hkv, -1, d)
    out, lse = _attend(c, q, [pages(s["k"], x) for x in _sources(c)], [pages(s["v"], x) for x in _sources(c)],
                       valid, _weights(c, pick.device))
    return dict(out=out, lse=lse, selected=chosen.to(torch.int32)[None])


PLAIN = dict(plan=_plain_plan, append=_plain_append, decode=_plain_decode, sparse=_plain_sparse)


# --------------------------------------------------------------------- the framework's
_contexts = {}


def _context(c):
    """The library context of a model's head layout: a program keeps one for all its requests."""
    from cross_layer_kv_shared_b200 import kvshare as K
    key = (c.get("q_heads", 1), c.get("kv_heads", 1), c.get("d", 64), c.get("dtype", "bf16"), c["batch"],
           c["max_blocks"] * c["page"], c.get("mix", False))
    if key not in _contexts:
        _, h = K.kvshare_create(1, key[0], key[1], key[2], K.KVS_F32 if key[3] == "f32" else K.KVS_BF16, key[4], key[5])
        if key[6]:
            K.kvshare_set_map(h, [(K.KVS_SRC_MIX, 0, 1)], [_mix_weights(key[1])])
        else:
            K.kvshare_set_map(h, [(K.KVS_SRC_SINGLE, 0, 0)])
        _contexts[key] = h
    return K, _contexts[key]


def _own(s):
    c = s["case"]
    if "context" not in s:                                       # the program's handle and view of the pool
        s["K"], s["context"] = _context(c)
        if c["op"] != "plan":
            s["pages"] = s["K"].Pages(k=s["k"], v=s["v"], block_table=s["block_table"], lengths=s["lengths"],
                                      bound_codes=s.get("bound_codes"), bound_scale=s.get("bound_scale"))
    K, h = s["K"], s["context"]
    if c["op"] == "plan":
        K.kvshare_plan_pages(h, s["lengths"], s["new_tokens"], s["block_table"], s["ring"], s["ring_state"],
                             s["lengths_out"], s["ring_state_out"], s["token_start"], s["slot_map"], s["position"],
                             page_size=c["page"])
        return dict(block_table=s["block_table"], ring=s["ring"], ring_state=s["ring_state_out"],
                    token_start=s["token_start"], lengths=s["lengths_out"], slot_map=s["slot_map"],
                    position=s["position"])
    if c["op"] == "append":
        K.kvshare_append_paged(h, s["pages"], 0, s["k_new"], s["v_new"], s["slot_map"])
        if not c["bounds"]:
            return dict(k=s["k"], v=s["v"])
        return dict(k=s["k"], v=s["v"], bounds=s["bound_codes"].float() * s["bound_scale"][..., None, None])
    if c["op"] == "decode":
        K.kvshare_decode_paged(h, s["pages"], s["q"], s["out"], s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    K.kvshare_select_pages(h, s["pages"], s["q"], s["selected"], first=1, last=1)
    K.kvshare_decode_paged(h, s["pages"], s["q"], s["out"], s["lse"], selected=s["selected"])
    return dict(out=s["out"], lse=s["lse"], selected=s["selected"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- work
def work(case):
    B, ps, P = case["batch"], case["page"], case["max_blocks"]
    if case["op"] == "plan":
        old, new = _new_tokens(case)
        fresh = sum(-(-(n + m) // ps) - -(-n // ps) for n, m in zip(old, new) if m > 0)
        back = sum(-(-n // ps) for n, m in zip(old, new) if m < 0)
        # lengths, counts in; starts and lengths out; pages moved between ring and table; two values a token out
        return dict(bytes=4 * (4 * B + 1 + 4 + 2 * (fresh + back)) + 8 * case["tokens"], flops=0)
    es = 2 if case["dtype"] == "bf16" else 4
    Hkv, Hq, d = case["kv_heads"], case["q_heads"], case["d"]
    if case["op"] == "append":
        old, new = _new_tokens(case)
        rows = sum(new)
        moved = 4 * rows * Hkv * d * es + 4 * case["tokens"]
        if case["bounds"]:
            touched = sum(-(-(n + m) // ps) - n // ps for n, m in zip(old, new) if m)
            earlier = sum(n % ps for n, m in zip(old, new) if m)     # rows the first page of a chunk already held
            moved += Hkv * (touched * (2 * d + 4) + earlier * d * es)
        return dict(bytes=moved, flops=0)
    nsrc = 2 if case["mix"] else 1
    lens = _lengths(case)
    fixed = B * Hq * (d * es + 4 * d + 4)                         # queries in, outputs and statistics out
    if case["op"] == "decode":
        tokens = sum(lens)
        moved = 2 * nsrc * tokens * Hkv * d * es + fixed + 4 * sum(-(-n // ps) for n in lens)
        return dict(bytes=moved, flops=4 * nsrc * tokens * Hq * d)
    held = [-(-n // ps) for n in lens]
    K = case["top"]
    # the last page is always kept, so the tokens read are known
    tokens = sum((min(K, p) - 1) * ps + n - (p - 1) * ps for n, p in zip(lens, held) if p)
    moved = 2 * nsrc * tokens * Hkv * d * es + fixed + nsrc * sum(held) * Hkv * (2 * d + 4) + 4 * B * Hkv * K + 4 * sum(held)
    return dict(bytes=moved, flops=4 * nsrc * tokens * Hq * d + 4 * nsrc * sum(held) * Hq * d)


# ------------------------------------------------------------------------------- exact
def _exact_rows(c, q, sources):
    """Softmax attention of q [g,d] over the sources' (k, v) [n,d], mixed by their weights, in 64 bits."""
    k = sum(wt * kk.double() for wt, kk, _ in sources)
    v = sum(wt * vv.double() for wt, _, vv in sources)
    z = (q.double() @ k.T) * c["d"] ** -0.5
    lse = torch.logsumexp(z, -1)
    return torch.softmax(z, -1) @ v, lse


def _exact_selection(s, b, j, weights):
    """The definition, a head and a page bound at a time, in whole numbers and IEEE 32-bit steps."""
    c = s["case"]
    ps, d, Hkv = c["page"], c["d"], c["kv_heads"]
    g = c["q_heads"] // Hkv
    n = _lengths(c)[b]
    held = -(-n // ps)
    ids = s["block_table"][b, :held].long()
    best = torch.full((held,), -math.inf, dtype=torch.float32, device=ids.device)
    for h in range(j * g, (j + 1) * g):
        q = s["q"][0, b, h].float()
        sq = q.abs().max() / 127
        qc = torch.round(q / sq).long() if sq > 0 else torch.zeros(d, dtype=torch.int64, device=ids.device)
        parts = []
        for src in _sources(c):
            codes = s["bound_codes"][src, ids, j].long()
            dot = torch.where(qc > 0, qc * codes[:, 0], qc * codes[:, 1]).sum(-1)
            parts.append(dot.float() * sq * s["bound_scale"][src, ids, j])
        score = parts[0] if len(parts) == 1 else weights[0] * parts[0] + weights[1] * parts[1]
        best = torch.maximum(best, score)
    rank = best.cpu().tolist()
    must = {0, held - 1}
    rest = sorted((p for p in range(held) if p not in must), key=lambda p: (-rank[p], p))
    return sorted((sorted(must) + rest)[: c["top"]])


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "plan":
        return None                                              # whole numbers only
    ps = c["page"]
    if op == "append":
        slot = s["slot_map"].tolist()
        k, v = s["k"].double(), s["v"].double()
        live = [i for i, x in enumerate(slot) if x >= 0]
        at = torch.tensor([slot[i] for i in live], device=k.device)
        src = torch.tensor(live, device=k.device)
        k[0, at // ps, :, at % ps] = s["k_new"][src].double()
        v[0, at // ps, :, at % ps] = s["v_new"][src].double()
        if not c["bounds"]:
            return dict(k=k, v=v)
        last = {}
        for i in live:
            last[slot[i] // ps] = max(last.get(slot[i] // ps, 0), slot[i] % ps + 1)
        bounds = torch.zeros(1, k.shape[1], c["kv_heads"], 2, c["d"], dtype=torch.float64, device=k.device)
        for page, rows in last.items():
            x = k[0, page, :, :rows]
            hi, lo = x.amax(1).float(), x.amin(1).float()
            scale = (torch.maximum(hi.abs(), lo.abs()).amax(-1, keepdim=True) / 127)
            bounds[0, page, :, 0] = (hi / scale).ceil().clamp(max=127).double() * scale.double()
            bounds[0, page, :, 1] = (lo / scale).floor().clamp(min=-127).double() * scale.double()
        return dict(k=k, v=v, bounds=bounds)
    B, Hkv, Hq, d = c["batch"], c["kv_heads"], c["q_heads"], c["d"]
    g = Hq // Hkv
    dev = s["q"].device
    out = torch.zeros(1, B, Hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((1, B, Hq), -math.inf, dtype=torch.float64, device=dev)
    w32 = torch.tensor(_mix_weights(Hkv), dtype=torch.float32, device=dev)
    chosen = torch.full((1, B, Hkv, c.get("top", 1)), -1, dtype=torch.int32, device=dev)
    for b, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        for j in range(Hkv):
            weights = [w32[j], 1 - w32[j]] if c["mix"] else [torch.ones((), device=dev)]
            blocks = list(range(-(-n // ps)))
            if op == "sparse":
                blocks = _exact_selection(s, b, j, weights)
                chosen[0, b, j, : len(blocks)] = torch.tensor(blocks, dtype=torch.int32, device=dev)
            ids = s["block_table"][b, torch.tensor(blocks, device=dev)].long()
            at = (torch.tensor(blocks, device=dev)[:, None] * ps + torch.arange(ps, device=dev)).reshape(-1) < n
            rows = lambda pool, x: pool[x, ids, j].reshape(-1, d)[at]  # noqa: E731
            sources = [(wt.double(), rows(s["k"], x), rows(s["v"], x)) for wt, x in zip(weights, _sources(c))]
            o, z = _exact_rows(c, s["q"][0, b, j * g:(j + 1) * g], sources)
            out[0, b, j * g:(j + 1) * g], lse[0, b, j * g:(j + 1) * g] = o, z
    return dict(out=out, lse=lse, selected=chosen) if op == "sparse" else dict(out=out, lse=lse)
