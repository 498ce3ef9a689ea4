"""Workloads of the library's language-model operators, with each operator's plain form.

Five operators, one ``op`` each: ``fwd`` and ``bwd`` are attention with a document or prefix mask, capped
scores and a distance bias, and its gradient; ``tree`` is attention of drafted tokens (a tree per request; one
token is ordinary decoding) over a paged key/value cache; ``tables`` builds block tables and slot maps from
request lengths; ``append`` writes new keys and values into the cache.  ``run`` calls the library where ``own``
is true and computes the plain form, in 32 bits, where it is false; ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt pair with bidirectional prefixes: latency
        attn("fwd", "fwd_short_prefix", "f16", 2, 8, 2, 131, 64, prefix=True),
        # prefix-LM batch with distance bias, grouped heads, the projection's (batch, seq, head) order
        attn("fwd", "fwd_prefix_alibi", "f16", 4, 32, 8, 2048, 128, prefix=True, alibi=True, bshd=True),
        # a packed row of documents with capped scores, bf16: pretraining at 8k
        attn("fwd", "fwd_docs_cap_8k", "bf16", 1, 32, 8, 8192, 128, docs=9, cap=30.0, bshd=True),
        # a short bidirectional batch of an encoder, odd length, every option but the prefix
        attn("bwd", "bwd_short_encoder", "f16", 2, 6, 3, 333, 64, causal=False, docs=3, cap=20.0, alibi=True),
        # the training step of a packed row of four documents
        attn("bwd", "bwd_docs_8k", "bf16", 1, 16, 4, 8192, 128, docs=4, bshd=True),
        # one request, one token: the latency of a decoding step
        tree("tree_single_token", "f16", 1, 1, 16, 4, 700, 64, 16),
        # a decoding batch: one token each, long contexts of unequal length
        tree("tree_decode_batch", "bf16", 48, 1, 32, 8, 8000, 128, 16),
        # speculative decoding: trees of up to 40 drafted tokens, capped scores
        tree("tree_draft_batch", "f16", 16, 40, 32, 8, 4096, 128, 64, cap=50.0),
        # the step of a decoding batch: one token each
        tables("tables_decode", 48, 1, 16, 600),
        # many requests with prompts among them
        tables("tables_prompts", 2048, 40, 16, 3000),
        # one decoding step's keys and values
        append("append_decode", "bf16", 48, 8, 128, 16),
        # a batch of prompts
        append("append_prompts", "f16", 24576, 8, 128, 64),
    ]


def attn(op, name, dtype, B, Hq, Hkv, S, D, causal=True, docs=0, prefix=False, cap=0.0, alibi=False, bshd=False, Skv=0):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "Skv": Skv or S, "D": D,
            "causal": causal or prefix, "docs": docs, "prefix": prefix, "cap": cap, "alibi": alibi, "bshd": bshd}


def tree(name, dtype, B, nodes, Hq, Hkv, ctx, D, page, cap=0.0, alibi=False):
    return {"name": name, "op": "tree", "dtype": dtype, "B": B, "nodes": nodes, "Hq": Hq, "Hkv": Hkv, "ctx": ctx,
            "D": D, "page": page, "cap": cap, "alibi": alibi}


def tables(name, B, new, page, ctx):
    return {"name": name, "op": "tables", "B": B, "new": new, "page": page, "ctx": ctx}


def append(name, dtype, N, H, D, page):
    return {"name": name, "op": "append", "dtype": dtype, "N": N, "H": H, "D": D, "page": page}


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm, odd ones among them."""
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "tree", "tree", "tables", "append"])
    dtype, D = rng.choice(["f16", "bf16"]), rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    cap, alibi = rng.choice([0.0, 0.0, 15.0, 50.0]), rng.random() < 0.3
    if op in ("fwd", "bwd"):
        B = size(1, 6)
        top = math.isqrt((2 ** 31 if op == "fwd" else 2 ** 30) * 3 // (4 * B * Hkv * g))
        S = size(65, min(8192, top))
        kind = rng.choice(["docs", "prefix", "causal", "full"])
        docs = min(size(1, 24), S // 16) if kind == "docs" else 0
        Skv = S + rng.randrange(-S // 3, S // 3) if kind in ("causal", "full") and rng.random() < 0.4 else S
        c = attn(op, "", dtype, B, Hkv * g, Hkv, S, D, kind != "full" and (kind != "docs" or rng.random() < 0.7), docs,
                 kind == "prefix", cap, alibi, rng.random() < 0.5, Skv)
    elif op == "tree":
        B = size(1, 64)
        nodes = rng.choice([1, 1, size(2, 64)])
        top = 2 ** 20 // (B * Hkv)
        c = tree("", dtype, B, nodes, Hkv * g, Hkv, size(nodes + 1, min(32000, max(nodes + 2, top))), D,
                 rng.choice([8, 16, 32, 64, 128]), cap, alibi)
    elif op == "tables":
        c = tables("", size(1, 2048), size(1, 40), rng.choice([8, 16, 32, 64, 128]), size(1, 3000))
    else:
        c = append("", dtype, size(1, 24576), Hkv, D, rng.choice([8, 16, 32, 64, 128]))
    del c["name"]
    return c


def lengths(count, total):
    """`count` unequal lengths of sum `total`, the same for every seed."""
    r = random.Random("%d %d" % (count, total))
    cuts = sorted(r.randrange(total + 1) for _ in range(count - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def doc_bounds(case):
    """Per batch row: document boundaries; what is behind the last one (up to an eighth of the row) is padding."""
    rows = []
    for b in range(case["B"]):
        n, at, row = case["docs"], 0, [0]
        for x in lengths(n, case["S"] - b * (case["S"] // 8) // max(1, case["B"] - 1)):
            at += x
            row.append(at)
        rows.append(row)
    return rows


def prefixes(case):
    """Per batch row: prefix length, a quarter of the keys and more or less."""
    return [[case["Skv"] * (b + 1) // (2 * case["B"] + 2)] for b in range(case["B"])]


def requests(case):
    """Per request: cached tokens with the drafted ones, and drafted ones."""
    r = random.Random("%d %d %d" % (case["B"], case["nodes"], case["ctx"]))
    T = [case["nodes"] if b == 0 else r.randint(1, case["nodes"]) for b in range(case["B"])]
    return [(case["ctx"] if b == 0 else r.randint(max(T[b], case["ctx"] // 2), case["ctx"])) for b in range(case["B"])], T


def steps(case):
    """Per request: cached tokens and new ones; one in thirty-two brings a prompt."""
    r = random.Random("%d %d %d" % (case["B"], case["new"], case["ctx"]))
    old = [r.randint(0, case["ctx"]) for _ in range(case["B"])]
    return old, [1 if case["new"] == 1 else r.randint(1, case["new"]) * (16 if b % 32 == 1 else 1) for b in range(case["B"])]


def intervals(case):
    """The first key and the end of the keys of each query, per batch row, as Python numbers."""
    S, Skv, out = case["S"], case["Skv"], []
    bounds, pre = doc_bounds(case) if case["docs"] else None, prefixes(case) if case["prefix"] else None
    for b in range(case["B"]):
        spans = list(zip(bounds[b], bounds[b][1:])) if bounds else [(0, Skv)]
        row = [(0, 0)] * S
        for lo, end in spans:
            for i in range(lo if bounds else 0, end if bounds else S):
                hi = end
                if case["causal"]:
                    hi = min(end, max(i + Skv - S + 1, pre[b][0] if pre else 0))
                row[i] = (lo, max(lo, hi))
        out.append(row)
    return out


def pairs(case):
    return sum(hi - lo for row in intervals(case) for lo, hi in row)


def work(case):
    if case["op"] in ("fwd", "bwd"):
        q, kv = case["B"] * case["Hq"] * case["S"], case["B"] * case["Hkv"] * case["Skv"]
        n = pairs(case) * case["Hq"]
        if case["op"] == "fwd":
            return {"bytes": 2 * case["D"] * (2 * q + 2 * kv) + 4 * q, "flops": 4 * case["D"] * n}
        return {"bytes": 2 * case["D"] * (4 * q + 4 * kv) + 4 * q, "flops": 10 * case["D"] * n}
    if case["op"] == "tree":
        kv, T = requests(case)
        return {"bytes": 4 * case["D"] * (case["Hkv"] * sum(kv) + case["Hq"] * sum(T)),
                "flops": 4 * case["D"] * case["Hq"] * sum(a * t for a, t in zip(kv, T))}
    if case["op"] == "tables":
        old, new = steps(case)
        pages = sum((a + n + case["page"] - 1) // case["page"] - (a + case["page"] - 1) // case["page"] for a, n in zip(old, new))
        return {"bytes": 4 * (4 * case["B"] + 2 * sum(new) + 2 * pages), "flops": 0}
    return {"bytes": 8 * case["N"] * case["H"] * case["D"] + 4 * case["N"], "flops": 0}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"fwd": prepare_attn, "bwd": prepare_attn, "tree": prepare_tree, "tables": prepare_tables,
            "append": prepare_append}[case["op"]](dict(case), g)


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare_attn(s, g):
    dt, D = DT[s["dtype"]], s["D"]

    def make(H, n, scale=1.0):
        if s["bshd"]:
            return randn(g, (s["B"], n, H, D), dt, scale).transpose(1, 2)
        return randn(g, (s["B"], H, n, D), dt, scale)

    s["Q"], s["K"], s["V"] = make(s["Hq"], s["S"], 1.5), make(s["Hkv"], s["Skv"]), make(s["Hkv"], s["Skv"])
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, s["Hq"] + 1, device="cuda") / s["Hq"]) if s["alibi"] else None
    s["bounds"] = ints(doc_bounds(s)) if s["docs"] else None
    s["prefixes"] = ints(prefixes(s)) if s["prefix"] else None
    s["O"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(s["B"], s["Hq"], s["S"], device="cuda")
    if s["op"] == "bwd":
        s["dO"] = make(s["Hq"], s["S"], 0.02)
        s["O"], s["lse"] = plain_fwd(s)   # what the forward pass has left
        if s["bshd"]:
            s["O"] = s["O"].transpose(1, 2).contiguous().transpose(1, 2)
        s["dQ"], s["dK"], s["dV"] = torch.empty_like(s["Q"]), torch.empty_like(s["K"]), torch.empty_like(s["V"])
    return s


def prepare_tree(s, g):
    dt, page = DT[s["dtype"]], s["page"]
    kv, T = requests(s)
    need = [(n + page - 1) // page for n in kv]
    pool = sum(need) + 7
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(s["B"], max(need) + 2, dtype=torch.int32, device="cuda")
    at = ints(need).cumsum(0) - ints(need)
    col = torch.arange(table.shape[1], device="cuda")
    table = torch.where(col[None] < ints(need)[:, None], order[(at[:, None] + col[None]).clamp(max=pool - 1)], table)
    s["table"], s["kv_lens"], s["N"] = table.contiguous(), ints(kv), sum(T)
    s["q_starts"] = ints([sum(T[:b]) for b in range(s["B"] + 1)])
    shape = (pool, page, s["Hkv"], s["D"])
    s["k_cache"], s["v_cache"] = randn(g, shape, dt), randn(g, shape, dt)
    s["Q"] = randn(g, (s["N"], s["Hq"], s["D"]), dt, 1.5)
    # a node's parent is one of the nodes before it, or the last cached token (-1)
    node = torch.cat([torch.arange(t, device="cuda") for t in T])
    u = torch.rand(s["N"], generator=g, device="cuda")
    s["parents"] = (torch.floor(u * (node + 1)) - 1).to(torch.int32)
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, s["Hq"] + 1, device="cuda") / s["Hq"]) if s["alibi"] else None
    s["O"] = torch.empty_like(s["Q"])
    return s


def prepare_tables(s, g):
    old, new = steps(s)
    page, B = s["page"], s["B"]
    have = [(a + page - 1) // page for a in old]
    want = [(a + n + page - 1) // page for a, n in zip(old, new)]
    pool = sum(want) + 11
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(want) + 1), -1, dtype=torch.int32, device="cuda")
    used = sum(have)
    at = ints(have).cumsum(0) - ints(have)
    col = torch.arange(table.shape[1], device="cuda")
    s["table"] = torch.where(col[None] < ints(have)[:, None], order[(at[:, None] + col[None]).clamp(max=pool - 1)], table).contiguous()
    s["free"], s["head"] = order[used:].contiguous(), ints([3])
    s["kv_lens"], s["new_lens"] = ints(old), ints(new)
    N = sum(new) + 5
    for name, n in (("kv_out", B), ("head_out", 1), ("q_starts", B + 1), ("positions", N), ("slots", N), ("counts", 3)):
        s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
    return s


def prepare_append(s, g):
    dt, page = DT[s["dtype"]], s["page"]
    pages = (s["N"] + page - 1) // page + 3
    s["k_cache"] = torch.zeros(pages, page, s["H"], s["D"], dtype=dt, device="cuda")
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    # keys and values side by side, as a fused projection leaves them
    kv = randn(g, (s["N"], 2 * s["H"], s["D"]), dt)
    s["K"], s["V"] = kv[:, :s["H"]], kv[:, s["H"]:]
    s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:s["N"]].to(torch.int32)
    if s["N"] > 4:
        s["slots"][-2:] = -1   # the padding of a step of fixed size
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    return RUN[s["op"]](s)


def run_fwd(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.masked_attention_fwd(s["Q"], s["K"], s["V"], s["O"], s["lse"], causal=s["causal"], softcap=s["cap"],
                                 alibi_slopes=s["slopes"], doc_bounds=s["bounds"], prefix_lens=s["prefixes"])
        return {"O": s["O"], "lse": s["lse"]}
    O, lse = plain_fwd(s)
    return {"O": O, "lse": lse}


def run_bwd(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.masked_attention_bwd(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["lse"], s["dQ"], s["dK"], s["dV"],
                                 causal=s["causal"], softcap=s["cap"], alibi_slopes=s["slopes"],
                                 doc_bounds=s["bounds"], prefix_lens=s["prefixes"])
        return {"dQ": s["dQ"], "dK": s["dK"], "dV": s["dV"]}
    dQ, dK, dV = plain_bwd(s)
    return {"dQ": dQ, "dK": dK, "dV": dV}


def run_tree(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.tree_attention_fwd(s["Q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["q_starts"],
                               s["parents"], s["O"], s["nodes"], softcap=s["cap"], alibi_slopes=s["slopes"])
        return {"O": s["O"]}
    return {"O": plain_tree(s)}


def run_tables(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.kv_block_tables(s["kv_lens"], s["new_lens"], s["free"], s["head"], s["table"], s["page"], s["kv_out"],
                            s["head_out"], s["q_starts"], s["positions"], s["slots"], s["counts"])
        return {k: s[k] for k in ("table", "kv_out", "head_out", "q_starts", "positions", "slots", "counts")}
    return plain_tables(s)


def run_append(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.kv_cache_append(s["K"], s["V"], s["slots"], s["k_cache"], s["v_cache"])
    else:
        keep = s["slots"] >= 0
        at = s["slots"][keep].long()
        s["k_cache"].view(-1, s["H"], s["D"])[at] = s["K"][keep]
        s["v_cache"].view(-1, s["H"], s["D"])[at] = s["V"][keep]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


RUN = {"fwd": run_fwd, "bwd": run_bwd, "tree": run_tree, "tables": run_tables, "append": run_append}


# ---------------------------------------------------------------------------- plain forms

def plain_mask(s):
    """(batch, S, Skv): whether the query sees the key."""
    i = torch.arange(s["S"], device="cuda")[None, :, None]
    j = torch.arange(s["Skv"], device="cuda")[None, None, :]
    see = torch.ones(s["B"], s["S"], s["Skv"], dtype=torch.bool, device="cuda")
    if s["causal"]:
        see = j <= i + (s["Skv"] - s["S"])
    if s["prefixes"] is not None:
        see = see | (j < s["prefixes"][:, 0, None, None])
    if s["bounds"] is not None:
        pos = torch.arange(s["S"], device="cuda")
        doc = (pos[None, :, None] >= s["bounds"][:, None, :]).sum(-1)   # 1 .. docs inside the documents
        doc = torch.where(doc <= s["docs"], doc, 0)
        see = see & (doc[:, :, None] == doc[:, None, :]) & (doc > 0)[:, :, None]
    return see.expand(s["B"], s["S"], s["Skv"])


def plain_scores(s):
    """Scores (batch, kv head, group, S, Skv) with the masked ones at -inf, and tanh of the capped ones."""
    g = s["Hq"] // s["Hkv"]
    q = s["Q"].float().reshape(s["B"], s["Hkv"], g, s["S"], s["D"])
    x = (q @ s["K"].float()[:, :, None].transpose(-1, -2)) * (1.0 / math.sqrt(s["D"]))
    t = None
    if s["cap"]:
        t = torch.tanh(x / s["cap"])
        x = s["cap"] * t
    if s["slopes"] is not None:
        i = torch.arange(s["S"], device="cuda")[:, None] + (s["Skv"] - s["S"])
        dist = (i - torch.arange(s["Skv"], device="cuda")[None, :]).abs().float()
        x = x - s["slopes"].reshape(1, s["Hkv"], g, 1, 1) * dist
    return torch.where(plain_mask(s)[:, None, None], x, -math.inf), t


def plain_fwd(s):
    x, _ = plain_scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p / torch.where(total > 0, total, 1.0)) @ s["V"].float()[:, :, None]
    lse = top[..., 0] + torch.log(total[..., 0])
    return o.reshape(s["B"], s["Hq"], s["S"], s["D"]).to(s["Q"].dtype), lse.reshape(s["B"], s["Hq"], s["S"])


def plain_bwd(s):
    g = s["Hq"] // s["Hkv"]
    shape = (s["B"], s["Hkv"], g, s["S"], s["D"])
    x, t = plain_scores(s)
    lse = s["lse"].reshape(shape[:-1])[..., None]
    p = torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0))   # masked scores are -inf: 0
    do, q, k = s["dO"].float().reshape(shape), s["Q"].float().reshape(shape), s["K"].float()[:, :, None]
    delta = (do * s["O"].float().reshape(shape)).sum(-1, keepdim=True)
    ds = p * (do @ s["V"].float()[:, :, None].transpose(-1, -2) - delta)
    if t is not None:
        ds = ds * (1 - t * t)
    ds = ds * (1.0 / math.sqrt(s["D"]))
    dq = (ds @ k).reshape(s["B"], s["Hq"], s["S"], s["D"])
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    return dq.to(s["Q"].dtype), dk.to(s["Q"].dtype), dv.to(s["Q"].dtype)


def plain_tree(s):
    B, T, H, g, D = s["B"], s["nodes"], s["Hkv"], s["Hq"] // s["Hkv"], s["D"]
    start, count = s["q_starts"][:-1].long(), (s["q_starts"][1:] - s["q_starts"][:-1]).long()
    node = torch.arange(T, device="cuda")
    row = (start[:, None] + node).clamp(max=s["N"] - 1)
    real = node < count[:, None]
    # sees[b, t, u]: u is t or above it in the tree
    up = (s["parents"][row][:, :, None] == node) & real[:, :, None]
    sees = torch.linalg.matrix_power(up.float() + torch.eye(T, device="cuda"), T) > 0
    depth = sees.sum(-1) - 1
    k = s["k_cache"][s["table"].long()].reshape(B, -1, H, D).permute(0, 2, 3, 1)[:, :, None].float()
    v = s["v_cache"][s["table"].long()].reshape(B, -1, H, D).permute(0, 2, 1, 3)[:, :, None].float()
    q = s["Q"].float()[row].reshape(B, T, H, g, D).permute(0, 2, 3, 1, 4)
    x = (q @ k) * (1.0 / math.sqrt(D))
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    j = torch.arange(x.shape[-1], device="cuda")
    ctx = s["kv_lens"].long() - count
    draft = (j[None] - ctx[:, None]).clamp(0, T - 1)                        # (B, keys)
    inside = (j[None] >= ctx[:, None]) & (j[None] < s["kv_lens"][:, None])
    see = torch.gather(sees, 2, draft[:, None].expand(B, T, -1)) & inside[:, None] | (j[None, None] < ctx[:, None, None])
    if s["slopes"] is not None:
        pos = torch.where(inside, ctx[:, None] + torch.gather(depth, 1, draft), j[None])
        dist = ((ctx[:, None] + depth)[:, :, None] - pos[:, None]).abs().float()
        x = x - s["slopes"].reshape(1, H, g, 1, 1) * dist[:, None, None]
    x = torch.where(see[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = ((p / p.sum(-1, keepdim=True)) @ v).permute(0, 3, 1, 2, 4).reshape(B, T, s["Hq"], D)
    req = torch.searchsorted(s["q_starts"][1:].contiguous(), torch.arange(s["N"], device="cuda", dtype=torch.int32), right=True)
    return o[req, torch.arange(s["N"], device="cuda") - start[req]].to(s["Q"].dtype)


def plain_tables(s):
    page, N = s["page"], s["slots"].shape[0]
    old, new = s["kv_lens"].long(), s["new_lens"].long()
    have, want = (old + page - 1) // page, (old + new + page - 1) // page
    start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    first = (want - have).cumsum(0) - (want - have)            # pages that requests before this one take
    col = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (col[None] >= have[:, None]) & (col[None] < want[:, None])
    pick = (s["head"].long() + first[:, None] + col[None] - have[:, None]).clamp(0, s["free"].shape[0] - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    n = torch.arange(N, device="cuda")
    req = torch.searchsorted(start[1:].contiguous(), n, right=True).clamp(max=s["B"] - 1)
    pos = old[req] + n - start[req]
    real = n < start[-1]
    slot = table[req, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    taken = (want - have).sum().reshape(1)
    i32 = torch.int32
    return {"table": table, "kv_out": (old + new).to(i32), "head_out": (s["head"] + taken).to(i32), "q_starts": start.to(i32),
            "positions": torch.where(real, pos, -1).to(i32), "slots": torch.where(real, slot, -1).to(i32),
            "counts": torch.cat([start[-1:], taken, torch.zeros_like(taken)]).to(i32)}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("fwd", "bwd"):
        return exact_attn(s)
    if s["op"] == "tree":
        return exact_tree(s)
    if s["op"] == "append":
        out = {}
        page_of, at = (s["slots"].long() // s["page"]), (s["slots"].long() % s["page"])
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        for name, new in (("k_cache", s["K"]), ("v_cache", s["V"])):
            out[name] = s[name].double()
            out[name][page_of[live], at[live]] = new[live].double()
        return out
    return None


def exact_attn(s):
    """Head by head; a query's keys are one interval."""
    B, Hq, g, S, Skv = s["B"], s["Hq"], s["Hq"] // s["Hkv"], s["S"], s["Skv"]
    if B * Hq * S * Skv * s["D"] > 6e11:
        return None
    scale = 1.0 / math.sqrt(s["D"])
    key, pos = torch.arange(Skv, device="cuda"), torch.arange(S, device="cuda", dtype=torch.float64) + (Skv - S)
    spans = torch.tensor(intervals(s), device="cuda")
    O = torch.zeros(B, Hq, S, s["D"], dtype=torch.float64, device="cuda")
    L = torch.zeros(B, Hq, S, dtype=torch.float64, device="cuda")
    dQ, dK, dV = torch.zeros_like(O), torch.zeros(s["K"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["K"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        out = ~((key >= spans[b, :, :1]) & (key < spans[b, :, 1:]))
        for h in range(Hq):
            q, k, v = s["Q"][b, h].double(), s["K"][b, h // g].double(), s["V"][b, h // g].double()
            z = torch.mm(q, k.T).mul_(scale)
            slope = 1.0
            if s["cap"]:
                z = torch.tanh(z / s["cap"])
                slope = 1.0 - z * z
                z = z * s["cap"]
            if s["slopes"] is not None:
                z -= s["slopes"][h].double() * (pos[:, None] - key[None].double()).abs()
            z.masked_fill_(out, -math.inf)
            L[b, h] = torch.logsumexp(z, 1)
            p = torch.exp(z - L[b, h][:, None]).nan_to_num_(0.0)
            O[b, h] = torch.mm(p, v)
            if s["op"] == "bwd":
                do = s["dO"][b, h].double()
                dV[b, h // g] += torch.mm(p.T, do)
                ds = p * (torch.mm(do, v.T) - (do * O[b, h]).sum(1, keepdim=True)) * slope * scale
                dQ[b, h] = torch.mm(ds, k)
                dK[b, h // g] += torch.mm(ds.T, q)
    return {"O": O, "lse": L} if s["op"] == "fwd" else {"dQ": dQ, "dK": dK, "dV": dV}


def exact_tree(s):
    """Request by request, the ancestors of each drafted token by walking up."""
    if s["D"] * s["Hq"] * sum(a * t for a, t in zip(*requests(s))) > 3e11:
        return None
    g, O = s["Hq"] // s["Hkv"], torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, parents = s["q_starts"].tolist(), s["kv_lens"].tolist(), s["parents"].tolist()
    for b in range(s["B"]):
        lo, T, n = starts[b], starts[b + 1] - starts[b], lens[b]
        out, where = torch.zeros(T, n, dtype=torch.bool), torch.arange(n, dtype=torch.float64).repeat(T, 1)
        out[:, n - T:] = True
        here = []
        for t in range(T):
            chain, u = [], t
            while u >= 0:
                chain.append(u)
                u = parents[lo + u]
            for d, u in enumerate(reversed(chain)):
                out[t, n - T + u], where[t, n - T + u] = False, n - T + d
            here.append(n - T + len(chain) - 1)
        out, where = out.cuda(), where.cuda()
        dist = torch.tensor(here, dtype=torch.float64, device="cuda")[:, None] - where
        at = s["table"][b, :(n + s["page"] - 1) // s["page"]].long()
        k = s["k_cache"][at].reshape(-1, s["Hkv"], s["D"])[:n].double()
        v = s["v_cache"][at].reshape(-1, s["Hkv"], s["D"])[:n].double()
        for h in range(s["Hq"]):
            z = torch.mm(s["Q"][lo:lo + T, h].double(), k[:, h // g].T) / math.sqrt(s["D"])
            if s["cap"]:
                z = s["cap"] * torch.tanh(z / s["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * dist
            O[lo:lo + T, h] = torch.mm(torch.softmax(z.masked_fill(out, -math.inf), 1), v[:, h // g])
    return {"O": O}
