"""Workloads of the operators around attention in training and serving steps, with each operator's plain form.

Five operators, one ``op`` each: ``rope_fwd`` and ``rope_bwd`` are the norms of queries and keys for each head with
the position rotation in the same pass, and its gradient; ``append`` writes a step's keys and values to the paged
cache with both applied on the way (to a cache of 16 bits, or to one of 4 bits, whose rows are then read back as a
chunked prompt does); ``tree4`` is attention of drafted tokens over the cache of 4 bits; ``verify`` keeps the drafted
tokens that the target's probabilities accept.  ``run`` calls the library where ``own`` is true and computes the plain
form, in 32 bits (64 for sums of probabilities), where it is false; ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
GROUP = 64                    # values of a row that share a scale and a minimum in the cache of 4 bits
EPS = 1e-6


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt before its attention: latency; rotation of neighbouring pairs
        rope("rope_fwd", "rope_fwd_short", "f16", 1, 16, 4, 33, 64, 64, interleaved=True),
        # a packed row of pretraining, as the fused projection leaves it, positions by document
        rope("rope_fwd", "rope_fwd_8k", "bf16", 1, 32, 8, 8192, 128, 128, docs=4),
        # a small fine-tuning batch of odd length, a part of each head rotated
        rope("rope_bwd", "rope_bwd_short", "f16", 2, 6, 3, 333, 64, 32),
        # the training step of the packed row
        rope("rope_bwd", "rope_bwd_8k", "bf16", 1, 32, 8, 8192, 128, 128, docs=4),
        # one decoding step of a batch: norms and rotation of its queries and keys, rows to the cache
        append("append_decode", "bf16", 48, 32, 8, 128, 16, 16, norm=True),
        # a batch of prompts into the cache of 4 bits and back
        append("append4_prompts", "f16", 24576, 0, 8, 128, 64, 4),
        # one request, one token: the latency of a decoding step
        tree4("tree4_single_token", "f16", 1, 1, 16, 4, 700, 64, 16),
        # a decoding batch: one token each, long contexts of unequal length
        tree4("tree4_decode_batch", "bf16", 48, 1, 32, 8, 8000, 128, 16),
        # speculative decoding: trees of up to 40 drafted tokens, capped scores
        tree4("tree4_draft_batch", "f16", 16, 40, 32, 8, 4096, 128, 64, cap=50.0),
        # one request with a chain of drafts from a smaller model
        verify("verify_chain_single", 1, 5, 32000, probs=True),
        # a batch of such chains, large vocabulary
        verify("verify_chain_batch", 64, 8, 128000, probs=True),
        # trees of drafts without probabilities (retrieved, or a head's best guesses), odd vocabulary
        verify("verify_tree_batch", 32, 24, 49999, tree=True),
    ]


def rope(op, name, dtype, B, Hq, Hkv, S, D, R, interleaved=False, docs=0, weights=True):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "D": D, "R": R,
            "interleaved": interleaved, "docs": docs, "weights": weights}


def append(name, dtype, N, Hq, Hkv, D, page, bits, norm=False, R=0):
    return {"name": name, "op": "append", "dtype": dtype, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R or D, "page": page,
            "bits": bits, "norm": norm}


def tree4(name, dtype, B, nodes, Hq, Hkv, ctx, D, page, cap=0.0):
    return {"name": name, "op": "tree4", "dtype": dtype, "B": B, "nodes": nodes, "Hq": Hq, "Hkv": Hkv, "ctx": ctx,
            "D": D, "page": page, "cap": cap}


def verify(name, B, nodes, V, probs=False, tree=False):
    return {"name": name, "op": "verify", "B": B, "nodes": nodes, "V": V, "probs": probs, "tree": tree}


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithm, odd ones among them."""
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope_fwd", "rope_bwd", "append", "tree4", "tree4", "verify", "verify"])
    dtype, D = rng.choice(["f16", "bf16"]), rng.choice([64, 128])
    Hkv, g = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    if op in ("rope_fwd", "rope_bwd"):
        B = size(1, 6)
        S = size(1, min(8192, 8192 * 40 * 128 // (B * Hkv * (g + 1) * D)))
        c = rope(op, "", dtype, B, Hkv * g, Hkv, S, D, rng.choice([D, D, D // 2, 16]), rng.random() < 0.3,
                 min(size(1, 8), S) if rng.random() < 0.5 else 0, rng.random() < 0.8)
    elif op == "append":
        bits = rng.choice([16, 4])
        c = append("", dtype, size(1, 24576), Hkv * g if bits == 16 and rng.random() < 0.5 else 0, Hkv, D,
                   rng.choice([8, 16, 32, 64, 128]), bits, bits == 16 and rng.random() < 0.6, rng.choice([D, D, D // 2]))
        c["N"] = min(c["N"], 24576 * 16 // (c["Hq"] + 2 * Hkv))
    elif op == "tree4":
        B = size(1, 64)
        nodes = rng.choice([1, 1, size(2, 64)])
        top = 2 ** 20 // (B * Hkv)
        c = tree4("", dtype, B, nodes, Hkv * g, Hkv, size(nodes + 1, min(32000, max(nodes + 2, top))), D,
                  rng.choice([8, 16, 32, 64, 128]), rng.choice([0.0, 0.0, 15.0, 50.0]))
    else:
        B, nodes = size(1, 64), size(1, 24)
        V = min(size(500, 150000), 64 * 8 * 128000 // (B * nodes))
        tree = rng.random() < 0.4
        c = verify("", B, nodes, V, not tree and rng.random() < 0.7, tree)
    del c["name"]
    return c


def lengths(count, total):
    """`count` unequal lengths of sum `total`, the same for every seed."""
    r = random.Random("%d %d" % (count, total))
    cuts = sorted(r.randrange(total + 1) for _ in range(count - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def requests(case):
    """Per request: cached tokens with the drafted ones, and drafted ones."""
    r = random.Random("%d %d %d" % (case["B"], case["nodes"], case["ctx"]))
    T = [case["nodes"] if b == 0 else r.randint(1, case["nodes"]) for b in range(case["B"])]
    return [(case["ctx"] if b == 0 else r.randint(max(T[b], case["ctx"] // 2), case["ctx"])) for b in range(case["B"])], T


def drafts(case):
    """Per request: nodes, the first one being the last token that is already decided."""
    r = random.Random("%d %d %d" % (case["B"], case["nodes"], case["V"]))
    return [case["nodes"] if b == 0 else r.randint((case["nodes"] + 1) // 2, case["nodes"]) for b in range(case["B"])]


def work(case):
    op = case["op"]
    if op in ("rope_fwd", "rope_bwd"):
        rows = case["B"] * case["S"] * (case["Hq"] + case["Hkv"])
        n = rows * case["D"]
        moved = 4 * n if op == "rope_fwd" else 6 * n
        return {"bytes": moved + 4 * case["R"] * min(case["S"], 8192) + 4 * case["B"] * case["S"], "flops": 10 * n}
    if op == "append":
        new = case["N"] * case["Hkv"] * case["D"]
        q = case["N"] * case["Hq"] * case["D"]
        stored = 4 * new if case["bits"] == 16 else new + new // 8 + 4 * new     # and the rows read back
        return {"bytes": 4 * new + 4 * q + stored + 4 * case["N"] * case["R"] + 8 * case["N"], "flops": 8 * (2 * new + q)}
    if op == "tree4":
        kv, T = requests(case)
        row = case["D"] // 2 + case["D"] // GROUP * 4
        return {"bytes": 2 * row * case["Hkv"] * sum(kv) + 4 * case["D"] * case["Hq"] * sum(T),
                "flops": 4 * case["D"] * case["Hq"] * sum(a * t for a, t in zip(kv, T))}
    # the row that the next token is drawn from, and the draft's row where it was refused there (most often)
    return {"bytes": 4 * case["V"] * case["B"] * (2 if case["probs"] and case["nodes"] > 1 else 1), "flops": 2 * case["V"] * case["B"]}


# ---------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"rope_fwd": prepare_rope, "rope_bwd": prepare_rope, "append": prepare_append, "tree4": prepare_tree4,
            "verify": prepare_verify}[case["op"]](dict(case), g)


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def rope_table(rows, R):
    """(rows, R): the cosines of R / 2 angles, then their sines."""
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def prepare_rope(s, g):
    dt, B, S, D, heads = DT[s["dtype"]], s["B"], s["S"], s["D"], s["Hq"] + s["Hkv"]
    # queries, keys and values side by side, (batch, seq, head): what the fused projection leaves
    scale = torch.exp2(torch.randn(heads + s["Hkv"], 1, generator=g, device="cuda"))
    qkv = (torch.randn(B, S, heads + s["Hkv"], D, generator=g, device="cuda") * scale).to(dt)
    s["Q"], s["K"] = qkv[:, :, :s["Hq"]].transpose(1, 2), qkv[:, :, s["Hq"]:heads].transpose(1, 2)
    w = lambda: (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if s["weights"] else None
    s["q_weight"], s["k_weight"], s["table"], s["positions"] = w(), w(), rope_table(max(S, 64), s["R"]), None
    if s["docs"]:
        one = torch.cat([torch.arange(n, device="cuda") for n in lengths(s["docs"], S)])
        s["positions"] = one.to(torch.int32)[None].expand(B, S).contiguous()
    s["Q_out"], s["K_out"] = (torch.empty(B, S, t.shape[1], D, dtype=dt, device="cuda").transpose(1, 2) for t in (s["Q"], s["K"]))
    if s["op"] == "rope_bwd":
        s["dQ_out"], s["dK_out"] = (randn(g, (B, S, t.shape[1], D), dt, 0.05).transpose(1, 2) for t in (s["Q"], s["K"]))
        dqkv = torch.empty_like(qkv)
        s["dQ"], s["dK"] = dqkv[:, :, :s["Hq"]].transpose(1, 2), dqkv[:, :, s["Hq"]:heads].transpose(1, 2)
        s["dq_weight"], s["dk_weight"] = (torch.empty(D, device="cuda") if s["weights"] else None for _ in range(2))
    return s


def prepare_append(s, g):
    dt, page, D, H, N = DT[s["dtype"]], s["page"], s["D"], s["Hkv"], s["N"]
    pages = (N + page - 1) // page + 3
    if s["bits"] == 16:
        s["caches"] = [torch.zeros(pages, page, H, D, dtype=dt, device="cuda") for _ in range(2)]
    else:
        s["caches"] = [empty_cache4(pages, page, H, D, dt) for _ in range(2)]
        s["read"] = [torch.zeros(N, H, D, dtype=dt, device="cuda") for _ in range(2)]
    # queries, keys and values side by side, as a fused projection leaves them; some channels of the keys are large
    loud = torch.exp2(0.7 * torch.randn(s["Hq"] + 2 * H, D, generator=g, device="cuda"))
    qkv = (torch.randn(N, s["Hq"] + 2 * H, D, generator=g, device="cuda") * loud).to(dt)
    s["Q"], s["K"], s["V"] = qkv[:, :s["Hq"]], qkv[:, s["Hq"]:s["Hq"] + H], qkv[:, s["Hq"] + H:]
    s["Q_out"] = torch.zeros(N, s["Hq"], D, dtype=dt, device="cuda")
    w = lambda: (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if s["norm"] else None
    s["q_weight"], s["k_weight"] = w(), w()
    rows = 8192
    s["table"] = rope_table(rows, s["R"])
    s["positions"] = torch.randint(rows, (N,), generator=g, device="cuda", dtype=torch.int32)
    s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:N].to(torch.int32)
    if N > 4:
        s["slots"][-2:] = -1      # the padding of a step of fixed size
        s["positions"][-2:] = -1
    return s


def empty_cache4(pages, page, H, D, dt):
    """Codes of two values a byte, and (scale, minimum) of each 64 values; a head's rows of a page lie together."""
    codes = torch.zeros(pages, H, page, D // 2, dtype=torch.uint8, device="cuda").transpose(1, 2)
    return codes, torch.zeros(pages, H, page, D // GROUP, 2, dtype=dt, device="cuda").transpose(1, 2)


def quantise(x, dt):
    """Codes (two values a byte) and (scale, minimum) of rows x, in 32 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale, low = ((high - low) * (1.0 / 15.0)).to(dt).float(), low.to(dt).float()
    code = torch.round((x - low) / torch.where(scale > 0, scale, 1.0)).clamp(0, 15)
    code = torch.where(scale > 0, code, 0.0).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([scale, low], -1).to(dt)


def dequantise(codes, params):
    """The values that codes stand for, in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return (code.unflatten(-1, (-1, GROUP)) * params[..., :1].float() + params[..., 1:].float()).flatten(-2)


def prepare_tree4(s, g):
    dt, page, H, D = DT[s["dtype"]], s["page"], s["Hkv"], s["D"]
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
    s["caches"] = []
    for _ in range(2):
        codes, params = empty_cache4(pool, page, H, D, dt)
        for lo in range(0, pool, 4096):    # in parts, to bound the memory
            c, p = quantise(torch.randn(min(4096, pool - lo), page, H, D, generator=g, device="cuda"), dt)
            codes[lo:lo + 4096], params[lo:lo + 4096] = c, p
        s["caches"].append((codes, params))
    s["Q"] = randn(g, (s["N"], s["Hq"], D), dt, 1.5)
    # a node's parent is one of the nodes before it, or the last cached token (-1)
    node = torch.cat([torch.arange(t, device="cuda") for t in T])
    u = torch.rand(s["N"], generator=g, device="cuda")
    s["parents"] = (torch.floor(u * (node + 1)) - 1).to(torch.int32)
    s["O"] = torch.empty_like(s["Q"])
    return s


def prepare_verify(s, g):
    T, V = drafts(s), s["V"]
    N = sum(T)
    s["N"], s["q_starts"] = N, ints([sum(T[:b]) for b in range(s["B"] + 1)])
    logits = torch.randn(N, V, generator=g, device="cuda") * 3.0
    s["target"] = torch.softmax(logits, -1)
    node = torch.cat([torch.arange(t, device="cuda") for t in T])
    first = torch.repeat_interleave(s["q_starts"][:-1].long(), ints(T).long())
    # below each node some later ones: any earlier node may be the parent, the root often
    up = torch.floor(torch.rand(N, generator=g, device="cuda") ** 2 * node).long() if s["tree"] else node - 1
    s["parents"] = up.to(torch.int32) if s["tree"] else None
    if s["tree"]:
        s["parents"][s["q_starts"][:-1].long()] = -1
    above = first + up.clamp(min=0)
    s["draft"] = None
    if s["probs"]:
        near = logits[above] + torch.randn(N, V, generator=g, device="cuda")      # a smaller model that knows the target a little
        s["draft"] = torch.softmax(near, -1)
        noise = torch.rand(N, V, generator=g, device="cuda").clamp(min=1e-20).log().neg()
        s["tokens"] = (s["draft"] / noise).argmax(-1).to(torch.int32)               # drawn from it
    else:
        # guesses: among the target's best tokens
        best = logits[above].topk(min(12, V), -1).indices
        pick = (torch.rand(N, generator=g, device="cuda") ** 2 * best.shape[1]).long()
        s["tokens"] = best[torch.arange(N, device="cuda"), pick].to(torch.int32)
    del logits
    s["u_accept"] = torch.rand(N, generator=g, device="cuda")
    s["u_sample"] = torch.rand(s["B"], generator=g, device="cuda")
    s["path"] = torch.zeros(s["B"], s["nodes"], dtype=torch.int32, device="cuda")
    s["counts"], s["next"] = (torch.zeros(s["B"], dtype=torch.int32, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------------------- one pass

def run(s):
    return RUN[s["op"]](s)


def run_rope_fwd(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.qk_norm_rope_fwd(s["Q"], s["K"], s["Q_out"], s["K_out"], cos_sin=s["table"], positions=s["positions"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"])
        return {"Q_out": s["Q_out"], "K_out": s["K_out"]}
    return {"Q_out": plain_rope(s, s["Q"], s["q_weight"]), "K_out": plain_rope(s, s["K"], s["k_weight"])}


def run_rope_bwd(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.qk_norm_rope_bwd(s["dQ_out"], s["dK_out"], s["Q"], s["K"], s["dQ"], s["dK"], cos_sin=s["table"],
                             positions=s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                             dq_weight=s["dq_weight"], dk_weight=s["dk_weight"], eps=EPS, interleaved=s["interleaved"])
        return {"dQ": s["dQ"], "dK": s["dK"], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}
    dq, dwq = plain_rope_bwd(s, s["dQ_out"], s["Q"], s["q_weight"])
    dk, dwk = plain_rope_bwd(s, s["dK_out"], s["K"], s["k_weight"])
    return {"dQ": dq, "dK": dk, "dq_weight": dwq, "dk_weight": dwk}


def run_append(s):
    k, v = s["caches"]
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        kw = dict(positions=s["positions"], cos_sin=s["table"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        if s["Hq"]:
            kw.update(Q=s["Q"], Q_out=s["Q_out"])
        if s["bits"] == 16:
            gsr.kv_cache_append_rope(s["K"], s["V"], s["slots"], k, v, **kw)
        else:
            gsr.kv_cache4_append_rope(s["K"], s["V"], s["slots"], k, v, **kw)
            gsr.kv_cache4_read(k, v, s["slots"], s["read"][0], s["read"][1])
    else:
        plain_append(s, k, v)
    out = {"k": k, "v": v} if s["bits"] == 16 else {"k": s["read"][0], "v": s["read"][1]}
    if s["Hq"]:
        out["Q_out"] = s["Q_out"]
    return out


def run_tree4(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.tree_attention4_fwd(s["Q"], s["caches"][0], s["caches"][1], s["table"], s["kv_lens"], s["q_starts"],
                                s["parents"], s["O"], s["nodes"], softcap=s["cap"])
        return {"O": s["O"]}
    return {"O": plain_tree4(s)}


def run_verify(s):
    if own:
        import tensor_core_gemm_multistage_gb300 as gsr
        gsr.verify_drafts(s["target"], s["tokens"], s["q_starts"], s["parents"], s["u_accept"], s["u_sample"], s["path"],
                          s["counts"], s["next"], draft_probs=s["draft"])
        return {"path": s["path"], "counts": s["counts"], "next": s["next"]}
    return plain_verify(s)


RUN = {"rope_fwd": run_rope_fwd, "rope_bwd": run_rope_bwd, "append": run_append, "tree4": run_tree4, "verify": run_verify}


# ---------------------------------------------------------------------------- plain forms

def rotate(y, cos, sin, R, interleaved, back=False):
    """Pairs of the first R columns turned by their angles (`back`: by the negative ones); cos, sin broadcast over y."""
    if interleaved:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
    if back:
        c, d = a * cos + b * sin, b * cos - a * sin
    else:
        c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, y[..., R:]], -1)


def angles(s):
    """cos and sin, (batch or 1, 1, seq, R / 2)."""
    R = s["R"]
    t = s["table"][:s["S"]][None] if s["positions"] is None else s["table"][s["positions"].long()]
    return t[:, None, :, :R // 2], t[:, None, :, R // 2:]


def plain_rope(s, x, w):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    return rotate(y, *angles(s), s["R"], s["interleaved"]).to(x.dtype)


def plain_rope_bwd(s, do, x, w):
    dy = rotate(do.float(), *angles(s), s["R"], s["interleaved"], back=True)
    if w is None:
        return dy.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    n = x32 * r
    dn = dy * w.float()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dy * n).sum((0, 1, 2))


def plain_append(s, k_cache, v_cache):
    R, at = s["R"], s["positions"].long()
    live = at >= 0
    t = s["table"][at.clamp(min=0)][:, None]
    cos, sin = t[..., :R // 2], t[..., R // 2:]

    def normed(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        return rotate(y, cos, sin, R, False)

    if s["Hq"]:
        s["Q_out"].copy_(torch.where(live[:, None, None], normed(s["Q"], s["q_weight"]), 0.0))
    slots = s["slots"][live].long()
    page, row = slots // s["page"], slots % s["page"]
    for cache, x, read in ((k_cache, normed(s["K"], s["k_weight"])[live], 0), (v_cache, s["V"].float()[live], 1)):
        if s["bits"] == 16:
            cache[page, row] = x.to(cache.dtype)
        else:
            cache[0][page, row], cache[1][page, row] = quantise(x, cache[1].dtype)
            s["read"][read][live] = dequantise(cache[0][page, row], cache[1][page, row]).to(cache[1].dtype)


def plain_tree4(s):
    B, T, H, g, D = s["B"], s["nodes"], s["Hkv"], s["Hq"] // s["Hkv"], s["D"]
    start, count = s["q_starts"][:-1].long(), (s["q_starts"][1:] - s["q_starts"][:-1]).long()
    node = torch.arange(T, device="cuda")
    row = (start[:, None] + node).clamp(max=s["N"] - 1)
    real = node < count[:, None]
    # sees[b, t, u]: u is t or above it in the tree
    up = (s["parents"][row][:, :, None] == node) & real[:, :, None]
    sees = torch.linalg.matrix_power(up.float() + torch.eye(T, device="cuda"), T) > 0
    (kc, kp), (vc, vp) = s["caches"]
    at = s["table"].long()
    k = dequantise(kc[at], kp[at]).reshape(B, -1, H, D).permute(0, 2, 3, 1)[:, :, None]
    v = dequantise(vc[at], vp[at]).reshape(B, -1, H, D).permute(0, 2, 1, 3)[:, :, None]
    q = s["Q"].float()[row].reshape(B, T, H, g, D).permute(0, 2, 3, 1, 4)
    x = (q @ k) * (1.0 / math.sqrt(D))
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    j = torch.arange(x.shape[-1], device="cuda")
    ctx = s["kv_lens"].long() - count
    draft = (j[None] - ctx[:, None]).clamp(0, T - 1)                        # (B, keys)
    inside = (j[None] >= ctx[:, None]) & (j[None] < s["kv_lens"][:, None])
    see = torch.gather(sees, 2, draft[:, None].expand(B, T, -1)) & inside[:, None] | (j[None, None] < ctx[:, None, None])
    x = torch.where(see[:, None, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = ((p / p.sum(-1, keepdim=True)) @ v).permute(0, 3, 1, 2, 4).reshape(B, T, s["Hq"], D)
    req = torch.searchsorted(s["q_starts"][1:].contiguous(), torch.arange(s["N"], device="cuda", dtype=torch.int32), right=True)
    return o[req, torch.arange(s["N"], device="cuda") - start[req]].to(s["Q"].dtype)


def plain_verify(s):
    B, T, N, V = s["B"], s["nodes"], s["N"], s["V"]
    start, count = s["q_starts"][:-1].long(), (s["q_starts"][1:] - s["q_starts"][:-1]).long()
    node = torch.arange(T, device="cuda")
    real = node < count[:, None]
    row = (start[:, None] + node).clamp(max=N - 1)                          # (B, T)
    up = (node - 1).expand(B, T) if s["parents"] is None else torch.where(real, s["parents"][row].long(), -1)
    up = torch.where(real, up, -1)
    token = s["tokens"][row].long()
    p = s["target"][torch.gather(row, 1, up.clamp(min=0)), token].double()  # of each node's token, after its parent
    u = s["u_accept"][row].double()
    sibling = (up[:, :, None] == up[:, None, :]) & (up >= 0)[:, :, None] & (node[None, :, None] > node[None, None, :])
    if s["draft"] is not None:                                              # chains: one child a node
        yes = u * s["draft"][row, token].double() < p
    else:
        twice = sibling & (token[:, :, None] == token[:, None, :])          # a token that an earlier sibling had
        gone = torch.where(sibling & ~(twice.any(-1))[:, None, :], p[:, None, :], 0.0).sum(-1)
        yes = ~twice.any(-1) & (u * (1.0 - gone) < p)
    yes = yes & (up >= 0)
    chosen = yes & ~(sibling & yes[:, None, :]).any(-1)
    chosen[:, 0] = real[:, 0]
    above = (up[:, :, None] == node) & real[:, :, None]
    sees = torch.linalg.matrix_power(above.float() + torch.eye(T, device="cuda"), T) > 0
    kept = ~(sees & ~chosen[:, None, :]).any(-1) & real                     # nodes whose whole way up was chosen
    depth = sees.sum(-1) - 1
    last = torch.where(kept, depth, -1).argmax(-1)                          # the deepest of them
    counts = kept.sum(-1) - 1
    path = torch.full((B, T + 1), -1, dtype=torch.int64, device="cuda")
    path.scatter_(1, torch.where(kept & (depth > 0), depth - 1, T), node.expand(B, T))
    dist = s["target"][torch.gather(row, 1, last[:, None])[:, 0]].double()
    below = (up == last[:, None]) & real                                    # refused children of the last node
    if s["draft"] is not None:
        child = below.float().argmax(-1)
        q = s["draft"][torch.gather(row, 1, child[:, None])[:, 0]].double()
        left = torch.where(below.any(-1)[:, None], (dist - q).clamp(min=0.0), dist)
    else:
        hit = torch.zeros(B, V + 1, dtype=torch.bool, device="cuda")
        hit.scatter_(1, torch.where(below, token, V), torch.ones_like(token, dtype=torch.bool))
        left = torch.where(hit[:, :V], 0.0, dist)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, dist)
    total = left.cumsum(-1)
    drawn = torch.searchsorted(total, s["u_sample"].double()[:, None] * total[:, -1:], right=True)[:, 0]
    i32 = torch.int32
    return {"path": path[:, :T].to(i32), "counts": counts.to(i32), "next": drawn.clamp(max=V - 1).to(i32)}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("rope_fwd", "rope_bwd"):
        return exact_rope(s)
    if s["op"] == "append":
        return exact_append(s)
    if s["op"] == "tree4":
        return exact_tree4(s)
    return None                                                             # whole numbers


def turned(x, w, table, R, interleaved):
    """Norm and rotation of rows x (..., D) in 64 bits: pairs as complex numbers; table (..., R) broadcasts over x."""
    if w is not None:
        x = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    head = x[..., :R].unflatten(-1, (R // 2, 2) if interleaved else (2, R // 2))
    head = head if interleaved else head.transpose(-1, -2)
    z = torch.view_as_complex(head.contiguous()) * torch.complex(table[..., :R // 2], table[..., R // 2:])
    z = torch.view_as_real(z)
    z = z if interleaved else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., R:]], -1)


def exact_rope(s):
    out = {}
    pos = torch.arange(s["S"], device="cuda").expand(s["B"], -1) if s["positions"] is None else s["positions"].long()
    table = s["table"].double()[pos][:, None]
    for n in ("Q", "K"):
        x, w = s[n].double().requires_grad_(), s[n.lower() + "_weight"]
        w = None if w is None else w.double().requires_grad_()
        y = turned(x, w, table, s["R"], s["interleaved"])
        if s["op"] == "rope_fwd":
            out[n + "_out"] = y.detach()
        else:
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["d%s_out" % n].double())
            out["d" + n] = grads[0]
            out["d%s_weight" % n.lower()] = None if w is None else grads[1]
    return out


def exact_append(s):
    live = s["positions"] >= 0
    slots = s["slots"][live].long()
    page, row = slots // s["page"], slots % s["page"]
    table = s["table"].double()[s["positions"].long().clamp(min=0)][:, None]
    w = lambda n: None if s[n] is None else s[n].double()
    k = turned(s["K"].double(), w("k_weight"), table, s["R"], False)
    out = {}
    for n, cache, x in (("k", s["caches"][0], k), ("v", s["caches"][1], s["V"].double())):
        if s["bits"] == 16:
            out[n] = cache.double()
            out[n][page, row] = x[live]
        else:
            # each 64 values on 16 equal steps from their minimum, both held in the cache's type
            x = x[live].unflatten(-1, (-1, GROUP))
            low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            held = lambda t: t.float().to(DT[s["dtype"]]).double()
            step, low = held((high - low) / 15), held(low)
            out[n] = torch.zeros(s["read"][0].shape, dtype=torch.float64, device="cuda")
            out[n][live] = (low + step * ((x - low) / step).round().clamp(0, 15)).flatten(-2)
    if s["Hq"]:
        out["Q_out"] = torch.where(live[:, None, None], turned(s["Q"].double(), w("q_weight"), table, s["R"], False), 0.0)
    return out


def exact_tree4(s):
    """Request by request, the ancestors of each drafted token by walking up."""
    if s["D"] * s["Hq"] * sum(a * t for a, t in zip(*requests(s))) > 3e11:
        return None
    g, O = s["Hq"] // s["Hkv"], torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    starts, lens, parents = s["q_starts"].tolist(), s["kv_lens"].tolist(), s["parents"].tolist()

    def rows(cache, at, n):
        codes, params = (t[at].flatten(0, 1)[:n] for t in cache)
        steps = torch.stack([codes % 16, codes // 16], -1).double().reshape(n, s["Hkv"], -1, GROUP)
        return (params[..., 1:].double() + steps * params[..., :1].double()).reshape(n, s["Hkv"], s["D"])

    for b in range(s["B"]):
        lo, T, n = starts[b], starts[b + 1] - starts[b], lens[b]
        out = torch.zeros(T, n, dtype=torch.bool)
        out[:, n - T:] = True
        for t in range(T):
            u = t
            while u >= 0:
                out[t, n - T + u] = False
                u = parents[lo + u]
        out = out.cuda()
        at = s["table"][b, :(n + s["page"] - 1) // s["page"]].long()
        k, v = rows(s["caches"][0], at, n), rows(s["caches"][1], at, n)
        for h in range(s["Hq"]):
            z = torch.mm(s["Q"][lo:lo + T, h].double(), k[:, h // g].T) / math.sqrt(s["D"])
            if s["cap"]:
                z = s["cap"] * torch.tanh(z / s["cap"])
            O[lo:lo + T, h] = torch.mm(torch.softmax(z.masked_fill(out, -math.inf), 1), v[:, h // g])
    return {"O": O}
