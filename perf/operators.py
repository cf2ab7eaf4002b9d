"""The operators of a batch that answers from one compressed prompt, as cases to be timed and
compared: page tables and slot maps, the append into pages, the attention of a decode step over
the shared prompt and each sequence's own pages, and the sampling of the next token.

With ``own`` false, ``run`` computes an operator in its plain form (elementary torch operations);
with ``own`` true it makes the call a user of the library makes.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of 8 sequences over 28 layers: every row grows by one token
        {"name": "pages, a decode step", "op": "pages", "B": 8, "L": 28, "page": 16, "mean": 4000, "mode": "step"},
        # admission: 64 prompts of ragged length enter empty tables, the slot of every token is wanted
        {"name": "pages, admission", "op": "pages", "B": 64, "L": 32, "page": 16, "mean": 512, "mode": "admit"},
        # a recompression: most rows shrink to a budget of their own, others are new or unchanged
        {"name": "pages, recompression", "op": "pages", "B": 256, "L": 32, "page": 32, "mean": 1000, "mode": "mixed"},
        # the rows of one decode step enter their pages (pages hold a head's tokens together)
        {"name": "append, a decode step", "op": "append", "T": 224, "Hkv": 4, "d": 128, "dtype": "bf16", "page": 16,
         "layout": "head"},
        # the rows of a prompt of 64k tokens enter pages that hold a token's heads together, from a
        # projection's output that holds q, k and v side by side
        {"name": "append, a prompt", "op": "append", "T": 65536, "Hkv": 8, "d": 128, "dtype": "bf16", "page": 64,
         "layout": "token"},
        # fp32 caches with heads of 64, a short prompt
        {"name": "attention, fp32 heads of 64", "op": "attn", "B": 3, "L": 2, "Hkv": 2, "G": 2, "d": 64, "dtype": "fp32",
         "P": 509, "own": 45, "page": 16, "merged": True},
        # one layer's call of a small batch: the latency of a step
        {"name": "attention, one layer", "op": "attn", "B": 16, "L": 1, "Hkv": 8, "G": 4, "d": 128, "dtype": "bf16",
         "P": 4096, "own": 200, "page": 32, "merged": False},
        # 8 sequences, 7 query heads per KV head, a merged prompt cache with its logit bias
        {"name": "attention, 7 heads a group", "op": "attn", "B": 8, "L": 28, "Hkv": 4, "G": 7, "d": 128, "dtype": "bf16",
         "P": 8200, "own": 700, "page": 16, "merged": True},
        # 64 sequences on a prompt of 64k tokens of which 20 % are kept
        {"name": "attention, 64 sequences", "op": "attn", "B": 64, "L": 32, "Hkv": 8, "G": 4, "d": 128, "dtype": "bf16",
         "P": 13107, "own": 256, "page": 64, "merged": False},
        # a decode step of 8 reasoning sequences: temperature 0.6, top-p 0.95
        {"name": "sampling, top-p", "op": "sample", "n": 8, "V": 152064, "dtype": "bf16", "mix": "top_p"},
        # a large batch whose requests carry parameters of their own
        {"name": "sampling, a mixed batch", "op": "sample", "n": 256, "V": 128256, "dtype": "bf16", "mix": "all"},
        # fp32 logits, an odd vocabulary, rows padded apart
        {"name": "sampling, fp32 odd", "op": "sample", "n": 5, "V": 32003, "dtype": "fp32", "mix": "all"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "append", "attn", "attn", "sample", "sample"])
    if op == "pages":
        return {"op": op, "B": _log(rng, 1, 256), "L": rng.randint(1, 32), "page": rng.choice([16, 32, 64, 128, 256]),
                "mean": _log(rng, 1, 1000), "mode": rng.choice(["step", "admit", "mixed"])}
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 65536), "Hkv": rng.randint(1, 8), "d": rng.choice([64, 128]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "page": rng.choice([16, 32, 64, 128, 256]),
                "layout": rng.choice(["head", "token"])}
    if op == "attn":
        c = {"op": op, "B": _log(rng, 1, 64), "L": _log(rng, 1, 32), "Hkv": rng.randint(1, 8), "G": rng.randint(1, 8),
             "d": rng.choice([64, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "bf16", "fp32"]),
             "P": _log(rng, 1, 32768), "own": _log(rng, 1, 1000), "page": rng.choice([16, 32, 64, 128, 256]),
             "merged": rng.random() < 0.5}
        if c["dtype"] == "fp32":               # fp32 caches serve small shapes
            c["L"], c["P"] = min(c["L"], 4), min(c["P"], 4000 + c["P"] % 97)
        top = work(listed()[8])
        while True:                            # no drawn case costs more than the largest listed one
            w = work(c)
            if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
                return c
            if c["L"] > 1:
                c["L"] -= 1
            else:
                c["B"] -= 1
    return {"op": op, "n": _log(rng, 1, 256), "V": _log(rng, 500, 152064), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
            "mix": rng.choice(["top_p", "all"])}


# Lengths belong to the case, values to the seed: work() and prepare() agree on them.

def _rng(case, tag):
    return random.Random("%s %s" % (tag, sorted((k, v) for k, v in case.items() if k != "name")))


def _prompt_lens(case):
    """Tokens of the prompt's compacted cache in each layer: P at most, budgets differ by layer."""
    r = _rng(case, "prompt")
    return [case["P"]] + [r.randint(max(1, (3 * case["P"]) // 4), case["P"]) for _ in range(case["L"] - 1)]


def _own_lens(case):
    """Tokens of each sequence's own pages in each layer: from none (just admitted) to twice the mean."""
    r = _rng(case, "own")
    out = []
    for b in range(case["B"]):
        n = 0 if r.random() < 0.1 else r.randint(1, 2 * case["own"])
        out.append([max(0, n - r.randint(0, n // 4)) for _ in range(case["L"])])
    return out


def _table_lens(case):
    """(held, wanted) tokens of every table row."""
    r = _rng(case, "pages")
    old, new = [], []
    for b in range(case["B"]):
        n = r.randint(0, 2 * case["mean"])
        kind = r.choice(["grow", "shrink", "shrink", "same", "new", "end"])
        for l in range(case["L"]):
            if case["mode"] == "step":
                a, z = n, n + 1
            elif case["mode"] == "admit":
                a, z = 0, n
            elif kind == "grow":
                a, z = n, n + r.randint(1, 64)
            elif kind == "shrink":
                a, z = n, r.randint(0, n)
            elif kind == "same":
                a, z = n, n
            elif kind == "new":
                a, z = 0, n
            else:
                a, z = n, 0
            old.append(a)
            new.append(z)
    return old, new


def _pages(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "pages":
        old, new = _table_lens(case)
        p = case["page"]
        taken = sum(max(0, _pages(z, p) - _pages(a, p)) for a, z in zip(old, new))
        freed = sum(max(0, _pages(a, p) - _pages(z, p)) for a, z in zip(old, new))
        slots = sum(max(0, z - a) for a, z in zip(old, new))
        # both lengths read; taken pages out of the ring into the tables, freed ones back; slots and starts
        return {"bytes": 4 * (3 * len(old) + 2 * taken + 2 * freed + slots), "flops": 4 * len(old) + slots}
    if op == "append":
        row = case["Hkv"] * case["d"] * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": case["T"] * (4 * row + 4), "flops": 0}
    if op == "attn":
        es = 2 if case["dtype"] == "bf16" else 4
        B, L, Hkv, G, d = (case[k] for k in ("B", "L", "Hkv", "G", "d"))
        P, O = sum(_prompt_lens(case)), sum(map(sum, _own_lens(case)))
        kv = 2 * Hkv * d * es * (P + O) + (4 * Hkv * P if case["merged"] else 0)
        qo = B * L * Hkv * G * (d * es + d * 4 + 4)
        return {"bytes": kv + qo, "flops": 4 * d * Hkv * G * (B * P + O)}
    return {"bytes": case["n"] * (case["V"] * (2 if case["dtype"] == "bf16" else 4) + 32), "flops": 4 * case["n"] * case["V"]}


# ----------------------------------------------------------------------------- the inputs

def _g(seed):
    return torch.Generator(device=DEV).manual_seed(1_000_003 * seed + 17)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _g(seed)
    return {"pages": _prep_pages, "append": _prep_append, "attn": _prep_attn, "sample": _prep_sample}[case["op"]](case, g)


def _prep_pages(case, g):
    old, new = _table_lens(case)
    p, rows = case["page"], len(old)
    held = sum(_pages(a, p) for a in old)
    taken = sum(max(0, _pages(z, p) - _pages(a, p)) for a, z in zip(old, new))
    n_pages = held + taken + 5 + (held + taken) // 8
    max_pages = max(1, max(_pages(max(a, z), p) for a, z in zip(old, new)))
    ids = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=DEV)
    have = (_i32(old) + p - 1) // p
    used = torch.arange(max_pages, device=DEV)[None, :] < have[:, None]
    table[used] = ids[:held]
    head = int(torch.randint(0, n_pages, (1,), device=DEV, generator=g))
    ring = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(n_pages - held, device=DEV)) % n_pages] = ids[held:]
    slots = sum(max(0, z - a) for a, z in zip(old, new))
    return {"op": "pages", "page": p, "lens": _i32(old), "lens_new": _i32(new), "table": table, "ring": ring,
            "state": _i32([head, n_pages - held]), "state_out": _i32([0, 0]), "lens_out": torch.empty_like(have),
            "slots": torch.empty(slots + 7, dtype=torch.int32, device=DEV),
            "slot_start": torch.empty(rows + 1, dtype=torch.int32, device=DEV)}


def _pool(case, n_pages, g):
    """A K and a V pool viewed as [page][head][token][d] in either memory layout."""
    H, p, d, dt = case["Hkv"], case["page"], case["d"], DTYPES[case["dtype"]]
    if case.get("layout", "head") == "head":
        return [torch.randn(n_pages, H, p, d, device=DEV, generator=g).to(dt) for _ in range(2)]
    return [torch.randn(n_pages, p, H, d, device=DEV, generator=g).to(dt).transpose(1, 2) for _ in range(2)]


def _prep_append(case, g):
    T, H, d, p = case["T"], case["Hkv"], case["d"], case["page"]
    dt = DTYPES[case["dtype"]]
    n_pages = _pages(T, p) + 3 + T // (4 * p)
    qkv = torch.randn(T, 3 * H * d, device=DEV, generator=g).to(dt)
    perm = torch.randperm(n_pages, device=DEV, generator=g)
    if case["layout"] == "head":              # one token a sequence: each in a page of its own where they suffice
        at = torch.arange(T, device=DEV)
        slots = perm[at % n_pages] * p + (at // n_pages + at % n_pages) % p
    else:                                     # a prompt's tokens in order, page after page
        at = torch.arange(T, device=DEV)
        slots = perm[at // p] * p + at % p
    slots = slots.to(torch.int32)
    slots[torch.rand(T, device=DEV, generator=g) < 0.02] = -1        # padding of a captured step
    K, V = _pool(case, n_pages, g)
    return {"op": "append", "k": qkv[:, H * d:2 * H * d].unflatten(1, (H, d)), "v": qkv[:, 2 * H * d:].unflatten(1, (H, d)),
            "K": K, "V": V, "slots": slots, "shape": (1, H, H, d)}


def _prep_attn(case, g):
    B, L, Hkv, G, d, p = (case[k] for k in ("B", "L", "Hkv", "G", "d", "page"))
    P, dt = case["P"], DTYPES[case["dtype"]]
    pl, ol = _prompt_lens(case), _own_lens(case)
    npg = [[_pages(n, p) for n in row] for row in ol]
    held, most = sum(map(sum, npg)), max(map(max, npg))
    n_pages = held + 3
    ids = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    table = torch.full((B, L, max(1, most)), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max(1, most), device=DEV) < _i32(npg)[..., None]] = ids[:held]
    K, V = _pool(case, n_pages, g)
    q = torch.randn(B, L, Hkv * G, d, device=DEV, generator=g).to(dt)
    Kp, Vp = [torch.empty(L, Hkv, P, d, dtype=dt, device=DEV) for _ in range(2)]
    for l in range(L):
        Kp[l] = torch.randn(Hkv, P, d, device=DEV, generator=g)
        Vp[l] = torch.randn(Hkv, P, d, device=DEV, generator=g)
    Kp[:, :, 0] *= 4                           # an attention sink
    R = None
    if case["merged"]:                         # most slots of a merged cache took nothing in
        R = 1 + 4 * torch.rand(L, Hkv, P, device=DEV, generator=g) * (torch.rand(L, Hkv, P, device=DEV, generator=g) < 0.2)
    return {"op": "attn", "shape": (L, Hkv * G, Hkv, d), "q": q, "Kp": Kp, "Vp": Vp, "R": R, "P": P, "lens_p": _i32(pl),
            "K": K, "V": V, "table": table, "lens": _i32(ol), "most": max(1, max(map(max, ol))),
            "o": torch.empty(B, L, Hkv * G, d, device=DEV), "lse": torch.empty(B, L, Hkv * G, device=DEV), "ws": None}


def _prep_sample(case, g):
    n, V, dt = case["n"], case["V"], DTYPES[case["dtype"]]
    buf = torch.empty(n, V + (5 if dt == torch.float32 else 0), dtype=dt, device=DEV)
    z = buf[:, :V]
    sig = torch.empty(n, device=DEV).uniform_(0.5, 4.0, generator=g)
    z.copy_(torch.randn(n, V, device=DEV, generator=g) * sig[:, None])
    some = torch.rand(n, device=DEV, generator=g)
    col = torch.randint(0, V, (n,), device=DEV, generator=g)
    z[torch.arange(n, device=DEV), col] += (12 * (some < 0.3)).to(dt)        # a confident step
    masked = torch.rand(n, 1, device=DEV, generator=g)
    drop = torch.rand(n, V, device=DEV, generator=g) < 0.5
    z.masked_fill_(drop & (masked > 0.9), float("-inf"))                      # a grammar's mask
    z.masked_fill_(drop & (masked < 0.05), torch.finfo(dt).min)
    r = torch.rand(4, n, device=DEV, generator=g)
    temp, top_p = torch.full((n,), 0.6, device=DEV), torch.full((n,), 0.95, device=DEV)
    top_k, min_p = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV)
    if case["mix"] == "all":
        temp = torch.where(r[0] < 0.15, torch.zeros_like(temp), 0.3 + r[0])
        top_p = torch.where(r[1] < 0.4, torch.ones_like(temp), 0.5 + 0.49 * r[1])
        top_k = torch.where(r[2] < 0.5, 0, (1 + (2000 ** r[2]).to(torch.int32))).to(torch.int32)
        min_p = torch.where(r[3] < 0.6, torch.zeros_like(temp), 0.2 * (r[3] - 0.6))
    u = torch.rand(n, device=DEV, generator=g)
    return {"op": "sample", "logits": z, "u": u, "temperature": temp, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "token": torch.empty(n, dtype=torch.int32, device=DEV), "logprob": torch.empty(n, device=DEV),
            "kept": torch.empty(n, dtype=torch.int32, device=DEV)}


# ----------------------------------------------------------------------------- one pass

def run(state):
    if own:
        from long_context_kv_obs_b200 import binding as B
        return {"pages": _own_pages, "append": _own_append, "attn": _own_attn, "sample": _own_sample}[state["op"]](B, state)
    return {"pages": _plain_pages, "append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[state["op"]](state)


def _own_pages(B, s):
    B.kvc_page_tables(lens=s["lens"], lens_new=s["lens_new"], table=s["table"], ring=s["ring"], state=s["state"],
                      page=s["page"], state_out=s["state_out"], lens_out=s["lens_out"], slots=s["slots"],
                      slot_start=s["slot_start"])
    return s["table"], s["ring"], s["state_out"], s["lens_out"], s["slots"], s["slot_start"]


def _plain_pages(s):
    lens, new, page, ring = s["lens"].long(), s["lens_new"].long(), s["page"], s["ring"]
    head, count = s["state"].long()
    n_pages, table = ring.numel(), s["table"]
    have, need = (lens + page - 1) // page, (new + page - 1) // page
    take, free = (need - have).clamp(min=0), (have - need).clamp(min=0)
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    # freed pages join the ring behind the free ones, taken ones leave at its head, both in row order
    fr = (col >= need[:, None]) & (col < have[:, None])
    freed = table[fr]
    ring[(head + count + torch.arange(freed.numel(), device=ring.device)) % n_pages] = freed
    tk = (col >= have[:, None]) & (col < need[:, None])
    total = take.sum()
    before = (take.cumsum(0) - take)[:, None] + (col - have[:, None])
    table.copy_(torch.where(tk, ring[(head + before.clamp(min=0)) % n_pages], table))
    state = torch.stack([(head + total) % n_pages, count - total + free.sum()]).to(torch.int32)
    # slots of the new tokens, row after row
    add = (new - lens).clamp(min=0)
    start = torch.cat([add.new_zeros(1), add.cumsum(0)])
    slots = torch.full_like(s["slots"], -1)
    row = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), add)
    at = lens[row] + torch.arange(row.numel(), device=lens.device) - start[row]
    slots[:row.numel()] = (table[row, at // page].long() * page + at % page).to(torch.int32)
    return table, ring, state, new.to(torch.int32), slots, start.to(torch.int32)


def _own_append(B, s):
    B.kvc_page_append(B.model(*s["shape"]), k=s["k"], v=s["v"], K=s["K"], V=s["V"], slots=s["slots"])
    return s["K"], s["V"]


def _plain_append(s):
    page = s["K"].shape[2]
    keep = torch.nonzero(s["slots"] >= 0).flatten()
    at = s["slots"][keep].long()
    s["K"][at // page, :, at % page] = s["k"][keep]
    s["V"][at // page, :, at % page] = s["v"][keep]
    return s["K"], s["V"]


def _own_attn(B, s):
    s["ws"] = B.kvc_prefix_decode_attn(
        B.model(*s["shape"]), q=s["q"], K_prefix=s["Kp"], V_prefix=s["Vp"], lens_prefix=s["lens_p"], max_len_prefix=s["P"],
        R=s["R"], K=s["K"], V=s["V"], table=s["table"], lens=s["lens"], max_len=s["most"], o=s["o"], lse=s["lse"],
        workspace=s["ws"])
    return s["o"], s["lse"]


def _plain_attn(s):
    L, Hq, Hkv, d = s["shape"]
    q, page = s["q"], s["K"].shape[2]
    B, G, P = q.shape[0], Hq // Hkv, s["P"]
    outs, lses = [], []
    for l in range(L):
        qh = q[:, l].float().view(B, Hkv, G, d).transpose(0, 1) * d ** -0.5               # [Hkv][B][G][d]
        sp = torch.matmul(qh.reshape(Hkv, B * G, d), s["Kp"][l].float().transpose(1, 2)).view(Hkv, B, G, P)
        if s["R"] is not None:
            sp = sp + torch.log(s["R"][l])[:, None, None, :]
        sp = sp.masked_fill(torch.arange(P, device=q.device) >= s["lens_p"][l], float("-inf"))
        t = s["table"][:, l].long().clamp(min=0)                                           # [B][pages]
        Ko = s["K"][t].float().permute(2, 0, 1, 3, 4).reshape(Hkv, B, -1, d)
        Vo = s["V"][t].float().permute(2, 0, 1, 3, 4).reshape(Hkv, B, -1, d)
        past = torch.arange(Ko.shape[2], device=q.device) >= s["lens"][:, l, None]         # [B][own]
        so = torch.matmul(qh, Ko.transpose(2, 3)).masked_fill(past[None, :, None, :], float("-inf"))
        m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
        ep, eo = torch.exp(sp - m), torch.exp(so - m)
        sums = ep.sum(-1) + eo.sum(-1)
        o = torch.matmul(ep.view(Hkv, B * G, P), s["Vp"][l].float()).view(Hkv, B, G, d) + torch.matmul(eo, Vo)
        outs.append((o / sums[..., None]).transpose(0, 1).reshape(B, Hq, d))
        lses.append((m[..., 0] + torch.log(sums)).transpose(0, 1).reshape(B, Hq))
    return torch.stack(outs, 1), torch.stack(lses, 1)


def _own_sample(B, s):
    B.kvc_sample(logits=s["logits"], u=s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                 min_p=s["min_p"], token=s["token"], logprob=s["logprob"], kept=s["kept"])
    return s["token"], s["logprob"], s["kept"]


def _plain_sample(s):
    # in 64 bits: sums of many tiny probabilities are compared with a border
    z, at = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    n, V = z.shape
    T = s["temperature"].double()[:, None]
    greedy = T <= 0
    x = (z - z[:, :1]) / torch.where(greedy, torch.ones_like(T), T)
    w = torch.exp(x)
    rank = torch.arange(V, device=z.device)[None, :]
    k = s["top_k"].long()[:, None]
    keep = (rank < torch.where(k > 0, k, V)) & (z > float("-inf"))
    w = w * keep
    mass = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    keep &= (p >= 1) | (mass - w < p * mass[:, -1:]) | (rank == 0)
    keep &= w >= s["min_p"].double()[:, None]
    keep &= ~greedy | (rank == 0)
    w = w * keep
    flat = torch.zeros_like(w).scatter_(1, at, w)                       # back in token order
    run_ = torch.cumsum(flat, 1)
    aim = s["u"].double()[:, None] * run_[:, -1:]
    token = (run_ <= aim).sum(1)
    prob = flat.gather(1, token[:, None]) / run_[:, -1:]
    return token.to(torch.int32), torch.log(prob)[:, 0].float(), keep.sum(1).to(torch.int32)


# ----------------------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    if case["op"] == "append":
        return None                            # rows are copied, nothing is computed
    s = prepare(case, seed)
    return {"pages": _exact_pages, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](s)


def _exact_pages(s):
    page, table, ring = s["page"], s["table"].cpu().numpy(), s["ring"].cpu().numpy()
    lens, new = s["lens"].tolist(), s["lens_new"].tolist()
    head, count = s["state"].tolist()
    n = len(ring)
    tail, slots, start = head + count, [], [0]
    for r, (a, z) in enumerate(zip(lens, new)):
        for j in range(_pages(a, page), _pages(z, page)):
            table[r, j] = ring[head % n]
            head, count = head + 1, count - 1
        start.append(start[-1] + max(0, z - a))
        if z > a:
            t = np.arange(a, z)
            slots.append(table[r, t // page] * page + t % page)
    for r, (a, z) in enumerate(zip(lens, new)):
        for j in range(_pages(z, page), _pages(a, page)):
            ring[tail % n] = table[r, j]
            tail, count = tail + 1, count + 1
    out = np.full(s["slots"].numel(), -1, np.int32)
    if slots:
        out[:start[-1]] = np.concatenate(slots)
    return tuple(_i32(x) for x in (table.tolist(), ring.tolist(), [head % n, count], new, out.tolist(), start))


def _exact_attn(s):
    L, Hq, Hkv, d = s["shape"]
    q, page = s["q"].double(), s["K"].shape[2]
    B, G = q.shape[0], Hq // Hkv
    o = torch.empty(B, L, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.empty(B, L, Hq, dtype=torch.float64, device=q.device)
    lens, lens_p = s["lens"].tolist(), s["lens_p"].tolist()
    for l in range(L):
        P = lens_p[l]
        kp, vp = s["Kp"][l, :, :P].double(), s["Vp"][l, :, :P].double()
        bias = None if s["R"] is None else torch.log(s["R"][l, :, :P].double())
        for b in range(B):
            n = lens[b][l]
            pg = s["table"][b, l, :_pages(n, page)].long()
            ko = s["K"][pg].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
            vo = s["V"][pg].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
            qq = q[b, l].view(Hkv, G, d)
            a = torch.einsum("hgd,hnd->hgn", qq, kp) / math.sqrt(d)
            if bias is not None:
                a = a + bias[:, None]
            a = torch.cat([a, torch.einsum("hgd,hnd->hgn", qq, ko) / math.sqrt(d)], 2)
            z = torch.logsumexp(a, 2)
            w = torch.exp(a - z[..., None])
            o[b, l] = (torch.einsum("hgn,hnd->hgd", w[..., :P], vp) + torch.einsum("hgn,hnd->hgd", w[..., P:], vo)).reshape(Hq, d)
            lse[b, l] = z.reshape(Hq)
    return o, lse


def _exact_sample(s):
    logits = s["logits"].float().cpu().numpy().astype(np.float64)
    par = [s[k].double().tolist() for k in ("temperature", "top_k", "top_p", "min_p", "u")]
    tok, lp, kept = [], [], []
    for z, T, k, p, mp, u in zip(logits, *par):
        best = int(np.argmax(z))
        if T <= 0:
            tok, lp, kept = tok + [best], lp + [0.0], kept + [1]
            continue
        w = np.exp((z - z[best]) / T)
        order = np.lexsort((np.arange(len(z)), -z))                    # value down, index up
        order = order[z[order] > -np.inf]
        if k > 0:
            order = order[:int(k)]
        c = np.cumsum(w[order].astype(np.longdouble))
        if p < 1:
            order = order[:1 + int(np.searchsorted(c, np.longdouble(p) * c[-1], side="left"))]
        order = order[w[order] >= mp]
        order.sort()
        c = np.cumsum(w[order].astype(np.longdouble))
        i = int(np.searchsorted(c, np.longdouble(u) * c[-1], side="right"))
        tok.append(int(order[i]))
        lp.append(float(np.log(w[order[i]] / c[-1])))
        kept.append(len(order))
    return _i32(tok), torch.tensor(lp, dtype=torch.float64, device=DEV), _i32(kept)
