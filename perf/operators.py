"""Cases of the cache operators behind drafted and bounded decoding.

Four operators around the K/V cache, each in a plain form (torch operations in
fp32) and, with ``own`` set, through the library's entry points:

tree     attention of a tree of drafted tokens over a cache: node t of sequence
         b sees the cached rows 0..kv_lens[b]-1 and, of the tree, its own
         ancestors and itself; the tree's keys and values are not in the cache.
observe  causal grouped-query attention that also adds, per cache slot and KV
         head, the softmax weight the slot received (one token or a chunk).
evict    keeps ``budget`` slots of every (layer, sequence, KV head): the most
         recent ``recent`` positions and the slots of the largest accumulated
         weight; kept rows below ``budget`` stay, the holes are filled by the
         kept rows behind it, in order.
commit   longest path of the drafted tree that the target's tokens confirm, and
         its rows' copy from the tree's buffers into every layer's cache.
"""
import math

import numpy
import torch

own = False

DEV = "cuda"
PAD = -2   # parent of a padding node

# heads, KV heads, head size, type: the head layouts of the named workloads,
# and others of the tests
HEADS = {
    "tiny_f32": (4, 2, 16, "f32"),
    "char_8l": (8, 4, 64, "bf16"),
    "gqa_768": (8, 2, 96, "bf16"),
    "llama3_8b": (32, 8, 128, "bf16"),
    "mqa_16": (16, 1, 128, "bf16"),
    "gqa_12": (12, 4, 64, "bf16"),
    "char_f32": (8, 4, 64, "f32"),
    "mha_32": (8, 8, 32, "bf16"),
}


def _case(name, op, heads, **kw):
    c = dict(name=name, op=op, heads=heads, batch=1, length=0, ragged=False)
    c.update(kw)
    return c


def listed():
    return [
        # A short draft behind a chat turn of a small model: latency only.
        _case("tree_small", "tree", "char_8l", nodes=4, length=250),
        # One user, a full 64-node draft at the 8B prefill length: the cache
        # has to be split over the whole GPU.
        _case("tree_8b_single", "tree", "llama3_8b", nodes=64, length=8192),
        # The 8B decode batch, each with a 16-node draft, at uneven lengths:
        # streams the caches.
        _case("tree_8b_batch", "tree", "llama3_8b", nodes=16, batch=32, length=8192, ragged=True),
        # Odd draft and lengths on the 96-wide heads.
        _case("tree_gqa", "tree", "gqa_768", nodes=33, batch=8, length=2047, ragged=True),
        # The smallest observed decode step: fp32 heads, one token each.
        _case("observe_f32", "observe", "tiny_f32", batch=4, seq=1, length=1000, ragged=True),
        # The 8B decode step, watched for eviction.
        _case("observe_8b_decode", "observe", "llama3_8b", batch=32, seq=1, length=8192),
        # The 8B prompt: accumulates the weights that the first eviction needs.
        _case("observe_8b_prompt", "observe", "llama3_8b", seq=8192),
        # A padded batch of prompts continuing a short cache, odd sizes.
        _case("observe_gqa_chunk", "observe", "gqa_768", batch=8, seq=517, length=130, ragged=True),
        # A small model's caches cut to a quarter, every layer at once.
        _case("evict_char", "evict", "char_8l", layers=8, batch=10, length=256, budget=64, recent=16, ragged=True),
        # 8B prompts of two sequences compacted into caches of an eighth.
        _case("evict_8b_prompt", "evict", "llama3_8b", layers=32, batch=2, length=8192, budget=1024, recent=256),
        # Acceptance in a small model: latency only.
        _case("commit_char", "commit", "char_8l", layers=8, batch=10, nodes=12, length=200, ragged=True),
        # Acceptance of 64-node drafts through the 8B stack.
        _case("commit_8b", "commit", "llama3_8b", layers=32, batch=8, nodes=64, length=440, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "observe", "observe", "evict", "commit"])
    heads = rng.choice(list(HEADS))
    h, kv, hd, dt = HEADS[heads]
    row = kv * hd * (4 if dt == "f32" else 2) * 2          # K and V bytes of one cached token
    cap_rows = (1 << 30) // row                            # rows of at most 1 GiB of cache
    if dt == "f32" or hd < 64:
        cap_rows = min(cap_rows, 1 << 16)                  # the small models
    batch = _log_int(rng, 1, 48)
    ragged = rng.random() < 0.5
    if op == "tree":
        nodes = _log_int(rng, 1, 128)
        most = min(cap_rows // batch, (1 << 30) // (batch * h * nodes) if nodes > 16 else 1 << 17, 65536)
        return dict(op=op, heads=heads, batch=batch, nodes=nodes, length=_log_int(rng, 1, max(2, most)),
                    ragged=ragged)
    if op == "observe":
        if rng.random() < 0.5:
            length = _log_int(rng, 1, max(2, min(cap_rows // batch, 65536)))
            return dict(op=op, heads=heads, batch=batch, seq=1, length=length, ragged=ragged)
        batch = min(batch, 8)
        pairs = 1 << 31 if dt == "bf16" and hd >= 64 else 1 << 24   # H * batch * seq * keys of the largest case
        seq = _log_int(rng, 2, 6000)
        seq = max(2, min(seq, int(math.sqrt(pairs / (h * batch)))))
        length = rng.randint(0, max(0, min(pairs // (h * batch * seq) - seq, 3000)))
        return dict(op=op, heads=heads, batch=batch, seq=seq, length=length, ragged=ragged)
    layers = rng.randint(1, 32)
    if op == "evict":
        batch = min(batch, 16)
        length = _log_int(rng, 8, max(16, min(cap_rows // (batch * layers), 16384)))
        budget = _log_int(rng, 1, length)
        return dict(op=op, heads=heads, layers=layers, batch=batch, length=length, budget=budget,
                    recent=rng.randint(0, budget), ragged=ragged)
    nodes = _log_int(rng, 1, 128)
    length = rng.randint(0, max(1, min(cap_rows // (2 * batch * layers), 600)))
    return dict(op=op, heads=heads, layers=layers, batch=batch, nodes=nodes, length=length, ragged=ragged)


# ------------------------------------------------------------------- inputs
def _lens(case, n=None, lo=None):
    """Lengths per sequence: all ``length``, or spread evenly from a quarter of it (ragged)."""
    n = case["length"] if n is None else n
    lo = n // 4 if lo is None else lo
    B = case["batch"]
    if not case["ragged"] or B == 1:
        return [n] * B
    return [lo + (n - lo) * (b + 1) // B for b in range(B)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _trees(case, g):
    """parents [B, T]: node 0 the root (the token sampled last), every other
    node below an earlier one; in a ragged batch the last nodes are padding."""
    B, T = case["batch"], case["nodes"]
    t = torch.arange(T, device=DEV)
    lo = (t - 1).clamp(min=0) // 3
    u = torch.rand((B, T), generator=g, device=DEV)
    par = (lo + (u * (t - lo).clamp(min=1)).floor()).to(torch.int32)
    par = torch.minimum(par, (t - 1).clamp(min=0).to(torch.int32))
    par[:, 0] = -1
    if case["ragged"]:
        live = torch.tensor(_lens(case, T, (T + 1) // 2), device=DEV)[:, None]
        par = torch.where(t[None] < live, par, torch.full_like(par, PAD))
    return par


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _layers(c):
    return [{n: c[n][i] for n in c} for i in range(len(c["k"]))]


def prepare(case, seed):
    g = _gen(seed)
    H, KV, hd, dts = HEADS[case["heads"]]
    dt = torch.float32 if dts == "f32" else torch.bfloat16
    B, op = case["batch"], case["op"]
    s = dict(case=case, lens=_ints(_lens(case)))
    if op == "tree":
        T, L = case["nodes"], case["length"]
        s["cap"] = L + T
        s["q"] = _randn(g, (B, T, H, hd), dt, 1.5)
        s["k"] = _randn(g, (B, s["cap"], KV, hd), dt)
        s["v"] = _randn(g, (B, s["cap"], KV, hd), dt)
        s["kn"] = _randn(g, (B, T, KV, hd), dt)
        s["vn"] = _randn(g, (B, T, KV, hd), dt)
        s["parents"] = _trees(case, g)
        s["out"] = torch.zeros((B, T, H * hd), dtype=dt, device=DEV)
    elif op == "observe":
        S, L = case["seq"], case["length"]
        cap = s["cap"] = L + S
        s["q"] = _randn(g, (B, S, H, hd), dt, 1.5)
        s["k"] = _randn(g, (B, cap, KV, hd), dt)
        s["v"] = _randn(g, (B, cap, KV, hd), dt)
        s["seq_lens"] = _ints(_lens(case, S, (S + 1) // 2))
        # the tokens the sequence has seen are more than its cache holds
        s["positions"] = s["lens"] * 3 + 1
        s["weights_in"] = torch.rand((B, KV, cap), generator=g, device=DEV) * 4.0
        s["weights"] = torch.zeros((B, KV, cap), device=DEV)
        s["slot_pos"] = torch.zeros((B, KV, cap), dtype=torch.int32, device=DEV)
        s["out"] = torch.zeros((B, S, H * hd), dtype=dt, device=DEV)
    elif op == "evict":
        L, budget = case["length"], case["budget"]
        n = case["layers"]
        s["positions"] = s["lens"] + 5
        # every layer's buffers are slices of one, as a program with one arena for its caches has them
        src = s["src"] = dict(k=_randn(g, (n, B, L, KV, hd), dt), v=_randn(g, (n, B, L, KV, hd), dt))
        # few slots hold most of the weight; some were never looked at
        w = torch.exp(2.5 * torch.randn((n, B, KV, L), generator=g, device=DEV))
        src["weights"] = torch.where(torch.rand(w.shape, generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
        # slots in the order that earlier evictions left them in
        half = s["lens"][:, None, None] // 2
        pos = torch.arange(L, dtype=torch.int32, device=DEV).expand(n, B, KV, L)
        src["slot_pos"] = torch.where(pos < half, half - 1 - pos, pos).to(torch.int32).contiguous()
        s["dst"] = dict(k=torch.zeros((n, B, budget, KV, hd), dtype=dt, device=DEV),
                        v=torch.zeros((n, B, budget, KV, hd), dtype=dt, device=DEV),
                        weights=torch.zeros((n, B, KV, budget), device=DEV),
                        slot_pos=torch.zeros((n, B, KV, budget), dtype=torch.int32, device=DEV))
        s["lens_out"] = torch.zeros_like(s["lens"])
    else:
        T, L = case["nodes"], case["length"]
        cap = s["cap"] = L + T
        n = case["layers"]
        s["kn"], s["vn"] = _randn(g, (n, B, T, KV, hd), dt), _randn(g, (n, B, T, KV, hd), dt)
        s["k"] = torch.zeros((n, B, cap, KV, hd), dtype=dt, device=DEV)
        s["v"] = torch.zeros((n, B, cap, KV, hd), dtype=dt, device=DEV)
        par = s["parents"] = _trees(case, g)
        draft = torch.randint(0, 128256, (B, T), generator=g, device=DEV, dtype=torch.int32)
        target = torch.randint(0, 128256, (B, T), generator=g, device=DEV, dtype=torch.int32)
        # most nodes' target token is drafted by one of their children (the last one's write stays)
        hit = torch.rand((B, T), generator=g, device=DEV) < 0.8
        pick = torch.where((par >= 0) & hit, par, torch.full_like(par, T)).to(torch.int64)
        order = torch.full((B, T + 1), -1, dtype=torch.int64, device=DEV)
        order.scatter_reduce_(1, pick, torch.arange(T, device=DEV).expand(B, T), "amax")
        child = order[:, :T]
        target = torch.where(child >= 0, draft.gather(1, child.clamp(min=0)), target)
        s["draft"], s["target"] = draft.contiguous(), target.contiguous()
        s["path"] = torch.zeros((B, T), dtype=torch.int32, device=DEV)
        s["accepted"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        s["next"] = torch.zeros((B,), dtype=torch.int32, device=DEV)
        s["lens_out"] = torch.zeros_like(s["lens"])
    if own:
        from llama_decoder_only_rmsnorm_b200 import binding as lib
        s["lib"] = lib
        cfg = s["cfg"] = lib.make_config(H * hd, H, KV, 4 * H * hd, dtype=dts)
        if op == "tree":
            n = lib.llama3_tree_workspace_size(cfg, B, case["nodes"], case["length"])
        elif op == "observe":
            n = lib.llama3_observe_workspace_size(cfg, B, case["seq"], case["length"])
        elif op == "evict":
            n = lib.llama3_evict_workspace_size(cfg, case["layers"], B, case["length"], case["budget"])
            s["src_c"] = lib.make_bounded_caches(_layers(s["src"]))
            s["dst_c"] = lib.make_bounded_caches(_layers(s["dst"]))
        else:
            n = 0
            s["node_c"] = lib.make_bounded_caches(_layers(dict(k=s["kn"], v=s["vn"])))
            s["cache_c"] = lib.make_bounded_caches(_layers(dict(k=s["k"], v=s["v"])))
        s["ws"] = torch.empty((max(n, 16),), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------- plain forms
def _reach(parents):
    """[B, T, T] bool: column a is an ancestor of row t, or t itself; and [B, T] whether t hangs on the cache."""
    B, T = parents.shape
    idx = torch.arange(T, device=parents.device)
    r = ((parents[:, :, None] == idx) | (idx[:, None] == idx)).to(torch.float32)
    n = 1
    while n < T:
        r = (torch.matmul(r, r) > 0).to(torch.float32)
        n *= 2
    dead = (torch.matmul(r, (parents < -1).to(torch.float32)[:, :, None]) > 0)[:, :, 0]
    return r > 0, ~dead


def _plain_tree(s):
    q, k, v, kn, vn, par, lens = (s[n] for n in ("q", "k", "v", "kn", "vn", "parents", "lens"))
    B, T, H, hd = q.shape
    KV, L = k.shape[2], s["case"]["length"]
    rep = H // KV
    seen, live = _reach(par)
    out = torch.empty((B, T, H * hd), dtype=q.dtype, device=q.device)
    step = max(1, (1 << 28) // max(1, H * T * (L + T) + KV * L * hd))
    for b in range(0, B, step):
        e = min(B, b + step)
        qq = q[b:e].float().view(e - b, T, KV, rep, hd).permute(0, 2, 3, 1, 4).reshape(e - b, KV, rep * T, hd)
        kk = torch.cat((k[b:e, :L], kn[b:e]), 1).float().permute(0, 2, 3, 1)
        vv = torch.cat((v[b:e, :L], vn[b:e]), 1).float().permute(0, 2, 1, 3)
        x = (torch.matmul(qq, kk) / math.sqrt(hd)).view(e - b, KV, rep, T, L + T)
        j = torch.arange(L, device=q.device)
        m = torch.cat(((j < lens[b:e, None])[:, None].expand(e - b, T, L), seen[b:e]), 2) & live[b:e, :, None]
        x = x.masked_fill(~m[:, None, None], float("-inf"))
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
        x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
        o = torch.matmul(x.view(e - b, KV, rep * T, L + T), vv)
        o = o.view(e - b, KV, rep, T, hd).permute(0, 3, 1, 2, 4).reshape(e - b, T, H * hd)
        out[b:e] = o.to(q.dtype)
    return out


def _plain_observe(s):
    q, k, v, lens, rows, pos = (s[n] for n in ("q", "k", "v", "lens", "seq_lens", "positions"))
    B, S, H, hd = q.shape
    KV, cap = k.shape[2], s["cap"]
    rep, pairs = H // KV, B * k.shape[2]
    qq = q.view(B, S, KV, rep, hd).permute(0, 2, 3, 1, 4).reshape(pairs, rep, S, hd)
    kk, vv = k.permute(0, 2, 1, 3).reshape(pairs, cap, hd), v.permute(0, 2, 1, 3).reshape(pairs, cap, hd)
    out = torch.empty((pairs, rep, S, hd), dtype=q.dtype, device=q.device)
    add = torch.empty((pairs, cap), device=q.device)
    j, t = torch.arange(cap, device=q.device), torch.arange(S, device=q.device)
    first, n = lens.repeat_interleave(KV), rows.repeat_interleave(KV)
    step = max(1, (1 << 28) // (rep * S * cap + cap * hd))
    for a in range(0, pairs, step):
        e = min(pairs, a + step)
        m = (j <= (first[a:e, None, None] + t[:, None])) & (t[:, None] < n[a:e, None, None])
        x = torch.matmul(qq[a:e].float().reshape(e - a, rep * S, hd), kk[a:e].float().transpose(1, 2))
        x = (x / math.sqrt(hd)).view(e - a, rep, S, cap).masked_fill(~m[:, None], float("-inf"))
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == float("-inf"), torch.zeros_like(top), top))
        x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
        out[a:e] = torch.matmul(x.reshape(e - a, rep * S, cap), vv[a:e].float()).view(e - a, rep, S, hd).to(q.dtype)
        add[a:e] = x.sum((1, 2))
    out = out.view(B, KV, rep, S, hd).permute(0, 3, 1, 2, 4).reshape(B, S, H * hd)
    first, n = lens[:, None, None], rows[:, None, None]
    old = torch.where(j < first, s["weights_in"], torch.zeros_like(s["weights_in"]))
    weights = torch.where(j < first + n, old + add.view(B, KV, cap), s["weights"])
    new = (j >= first) & (j < first + n)
    slot_pos = torch.where(new, (pos[:, None, None] + j - first).to(torch.int32), s["slot_pos"])
    return {"out": out, "weights": weights, "slot_pos": slot_pos}


def _plain_evict(s):
    case, lens = s["case"], s["lens"]
    budget, L = case["budget"], case["length"]
    j = torch.arange(L, device=lens.device)
    i = torch.arange(budget, device=lens.device)
    n = lens[:, None, None]
    left = lens.clamp(max=budget)
    res = {n: s["dst"][n].clone() for n in s["dst"]}
    for src, dst, new in zip(_layers(s["src"]), _layers(s["dst"]), _layers(res)):
        recent = src["slot_pos"] >= s["positions"][:, None, None] - case["recent"]
        key = torch.where(recent, torch.full_like(src["weights"], float("inf")), src["weights"])
        key = torch.where(j < n, key, torch.full_like(key, float("-inf")))
        best = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
        keep = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, best, True) & (j < n)
        hole = ~keep[..., :budget]
        tail = keep & (j >= budget)
        rank = torch.cumsum(tail, -1) - 1
        where = torch.zeros(key.shape[:2] + (L + 1,), dtype=torch.int64, device=key.device)
        where.scatter_(-1, torch.where(tail, rank, torch.full_like(rank, L)), j.expand_as(key))
        fill = where.gather(-1, (torch.cumsum(hole, -1) - 1).clamp(min=0))
        take = torch.where(hole, fill, i.expand_as(fill))
        valid = i < left[:, None, None]
        rows = take.permute(0, 2, 1)[..., None].expand(-1, -1, -1, src["k"].shape[-1])
        ok = valid.permute(0, 2, 1)[..., None]
        new["k"].copy_(torch.where(ok, src["k"].gather(1, rows), dst["k"]))
        new["v"].copy_(torch.where(ok, src["v"].gather(1, rows), dst["v"]))
        new["weights"].copy_(torch.where(valid, src["weights"].gather(-1, take), dst["weights"]))
        new["slot_pos"].copy_(torch.where(valid, src["slot_pos"].gather(-1, take), dst["slot_pos"]))
    return {**res, "lens": left}


def _plain_commit(s):
    par, draft, target, lens = s["parents"], s["draft"], s["target"], s["lens"]
    B, T = par.shape
    idx = torch.arange(T, device=par.device)
    up = par.clamp(min=0).to(torch.int64)
    said = (draft == target.gather(1, up)) & (par >= 0)
    twin = (par[:, :, None] == par[:, None, :]) & (draft[:, :, None] == draft[:, None, :]) & (idx < idx[:, None])
    good = (said & ~twin.any(-1)) | ((idx == 0) & (par == -1))
    seen, _ = _reach(par)
    path = ~(seen & ~good[:, None, :]).any(-1)
    count = path.sum(-1).to(torch.int32)
    order = torch.sort(torch.where(path, idx, torch.full_like(idx, T)), -1).values
    last = torch.where(path, idx, torch.full_like(idx, -1)).amax(-1)
    nxt = torch.where(last >= 0, target.gather(1, last.clamp(min=0)[:, None])[:, 0], torch.full_like(count, -1))
    order = torch.where(order < T, order, torch.full_like(order, -1))
    slot = lens[:, None].to(torch.int64) + idx
    row = torch.arange(B, device=par.device)[:, None]
    ok = (idx < count[:, None])[..., None, None]
    take = order.clamp(min=0)
    for n in range(len(s["k"])):
        for cache, nodes in ((s["k"][n], s["kn"][n]), (s["v"][n], s["vn"][n])):
            cache[row, slot] = torch.where(ok, nodes[row, take], cache[row, slot])
    return {"path": order.to(torch.int32), "accepted": count, "next": nxt, "lens": lens + count,
            "k": s["k"], "v": s["v"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"tree": _plain_tree, "observe": _plain_observe, "evict": _plain_evict,
                "commit": _plain_commit}[op](s)
    lib, case, cfg, ws = s["lib"], s["case"], s["cfg"], s["ws"]
    if op == "tree":
        lib.llama3_attention_tree(cfg, s["q"], s["k"], s["v"], s["cap"], s["lens"], case["length"], s["kn"], s["vn"],
                                  s["parents"], case["batch"], case["nodes"], s["out"], ws, ws.numel())
        return s["out"]
    if op == "observe":
        lib.llama3_attention_observed(cfg, s["q"], s["k"], s["v"], s["cap"], case["batch"], case["seq"], s["lens"],
                                      s["seq_lens"], case["length"], s["out"], s["weights_in"], s["weights"],
                                      s["positions"], s["slot_pos"], ws, ws.numel())
        return {"out": s["out"], "weights": s["weights"], "slot_pos": s["slot_pos"]}
    if op == "evict":
        lib.llama3_cache_evict(cfg, s["src_c"], case["length"], s["dst_c"], case["budget"], case["batch"], s["lens"],
                               case["length"], case["budget"], case["recent"], s["positions"], s["lens_out"], ws,
                               ws.numel())
        return {**s["dst"], "lens": s["lens_out"]}
    lib.llama3_tree_accept(s["draft"], s["target"], s["parents"], case["batch"], case["nodes"], s["lens"],
                           s["path"], s["accepted"], s["next"], s["lens_out"])
    lib.llama3_tree_commit(cfg, s["node_c"], s["cache_c"], s["cap"], case["batch"], case["nodes"], s["path"],
                           s["accepted"], s["lens_out"])
    return {"path": s["path"], "accepted": s["accepted"], "next": s["next"], "lens": s["lens_out"],
            "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------------- work
def work(case):
    H, KV, hd, dts = HEADS[case["heads"]]
    es = 4 if dts == "f32" else 2
    B, op = case["batch"], case["op"]
    lens = _lens(case)
    row = KV * hd * es                                   # one token's K (or V)
    if op == "tree":
        T = case["nodes"]
        live = _lens(case, T, (T + 1) // 2) if case["ragged"] else [T] * B
        return {"bytes": 2 * (sum(lens) + sum(live)) * row + 2 * B * T * H * hd * es + 4 * B * (T + 1),
                "flops": sum(4 * H * hd * n * (x + 1) for n, x in zip(live, lens))}
    if op == "observe":
        S = case["seq"]
        rows = _lens(case, S, (S + 1) // 2)
        keys = sum(a + b for a, b in zip(lens, rows))
        pairs = sum(n * x + n * (n + 1) // 2 for n, x in zip(rows, lens))
        return {"bytes": 2 * keys * row + 2 * B * S * H * hd * es + (sum(lens) + keys) * KV * 4,
                "flops": 4 * H * hd * pairs}
    if op == "evict":
        left = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": case["layers"] * (sum(lens) * KV * 8 + left * (4 * row + KV * 8)), "flops": 0}
    # about half the depth of the tree is confirmed
    deep = max(1, int(math.log2(case["nodes"] + 1)))
    return {"bytes": B * case["nodes"] * 16 + case["layers"] * B * deep * 4 * row, "flops": 0}


# --------------------------------------------------------------------- exact
def _chains(parents):
    """Per sequence and node: the node's chain down to its root, or None where it does not hang on the cache."""
    res = []
    for p in parents.tolist():
        chains = []
        for t in range(len(p)):
            c, chain = t, []
            while c >= 0:
                chain.append(c)
                c = p[c]
            chains.append(sorted(chain) if c == -1 else None)
        res.append(chains)
    return res


def exact(case, seed):
    s = prepare(case, seed)
    H, KV, hd, _ = HEADS[case["heads"]]
    rep, B, op = H // KV, case["batch"], case["op"]
    scale = 1.0 / math.sqrt(hd)
    lens = s["lens"].tolist()
    if op == "tree":
        T = case["nodes"]
        out = torch.zeros((B, T, H, hd), dtype=torch.float64, device=DEV)
        for b, chains in enumerate(_chains(s["parents"])):
            alive = [t for t in range(T) if chains[t] is not None]
            if not alive:
                continue
            n = lens[b]
            see = torch.full((len(alive), n + T), -float("inf"), dtype=torch.float64, device=DEV)
            see[:, :n] = 0.0
            at = torch.tensor([(i, n + a) for i, t in enumerate(alive) for a in chains[t]], device=DEV)
            see[at[:, 0], at[:, 1]] = 0.0
            rows = torch.tensor(alive, device=DEV)
            for g in range(KV):
                kk = torch.cat((s["k"][b, :n, g], s["kn"][b, :, g])).double()
                vv = torch.cat((s["v"][b, :n, g], s["vn"][b, :, g])).double()
                for h in range(g * rep, (g + 1) * rep):
                    p = torch.softmax(s["q"][b, rows, h].double() @ kk.T * scale + see, -1)
                    out[b, rows, h] = p @ vv
        return out.view(B, T, H * hd)
    if op == "observe":
        S, cap = case["seq"], s["cap"]
        rows = s["seq_lens"].tolist()
        out = torch.zeros((B, S, H, hd), dtype=torch.float64, device=DEV)
        weights, slot_pos = s["weights"].double(), s["slot_pos"].clone()
        for b in range(B):
            n, x = rows[b], lens[b]
            slot_pos[b, :, x:x + n] = int(s["positions"][b]) + torch.arange(n, dtype=torch.int32, device=DEV)
            weights[b, :, :x] = s["weights_in"][b, :, :x].double()
            weights[b, :, x:x + n] = 0.0
            for g in range(KV):
                kk, vv = s["k"][b, :x + n, g].double(), s["v"][b, :x + n, g].double()
                for t in range(0, n, 1024):
                    e = min(n, t + 1024)
                    hide = torch.ones((e - t, x + n), dtype=torch.bool, device=DEV).triu(x + t + 1)
                    for h in range(g * rep, (g + 1) * rep):
                        a = (s["q"][b, t:e, h].double() @ kk.T * scale).masked_fill(hide, -float("inf"))
                        p = torch.softmax(a, -1)
                        out[b, t:e, h] = p @ vv
                        weights[b, g, :x + n] += p.sum(0)
        return {"out": out.view(B, S, H * hd), "weights": weights, "slot_pos": slot_pos}
    if op == "evict":
        res = {n: s["dst"][n].clone() for n in s["dst"]}
        for src, new in zip(_layers(s["src"]), _layers(res)):
            w, pos = src["weights"].cpu().numpy(), src["slot_pos"].cpu().numpy()
            for b in range(B):
                n, left = lens[b], min(lens[b], case["budget"])
                for g in range(KV):
                    old = pos[b, g, :n] < int(s["positions"][b]) - case["recent"]
                    order = numpy.lexsort((numpy.arange(n), numpy.where(old, -w[b, g, :n], 0.0), old))
                    kept = numpy.sort(order[:left])
                    take = numpy.arange(left)
                    take[~numpy.isin(take, kept)] = kept[kept >= left]
                    take = torch.from_numpy(take).to(DEV)
                    new["k"][b, :left, g] = src["k"][b, take, g]
                    new["v"][b, :left, g] = src["v"][b, take, g]
                    new["weights"][b, g, :left] = src["weights"][b, g, take]
                    new["slot_pos"][b, g, :left] = src["slot_pos"][b, g, take]
        res = {n: res[n].double() if res[n].is_floating_point() else res[n] for n in res}
        return {**res, "lens": _ints([min(n, case["budget"]) for n in lens])}
    T = case["nodes"]
    par, draft, target = (s[n].tolist() for n in ("parents", "draft", "target"))
    path, count, nxt = [], [], []
    for b in range(B):
        cur, p = (0, [0]) if par[b][0] == -1 else (None, [])
        while cur is not None:
            kids = [c for c in range(T) if par[b][c] == cur and draft[b][c] == target[b][cur]]
            cur = kids[0] if kids else None
            p += kids[:1]
        nxt.append(target[b][p[-1]] if p else -1)
        count.append(len(p))
        path.append(p + [-1] * (T - len(p)))
    for n in range(case["layers"]):
        for b in range(B):
            for i in range(count[b]):
                s["k"][n][b, lens[b] + i] = s["kn"][n][b, path[b][i]]
                s["v"][n][b, lens[b] + i] = s["vn"][n][b, path[b][i]]
    return {"path": _ints(path), "accepted": _ints(count), "next": _ints(nxt),
            "lens": _ints([a + c for a, c in zip(lens, count)]),
            "k": s["k"].double(), "v": s["v"].double()}
