"""What is measured of the decode operators around the MoE and GatedDeltaNet steps: the rotation and append of keys
and values to a paged cache, attention over that cache with a prefix that the whole batch shares, and the choice of
the next token.

``own`` false: plain forms in elementary torch operations; true: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence decoding one token: the latency of a single launch
        _append("append 1 token", T=1, seqs=1, n_kv=8, group=4, D=128, rd=128, axes=1, adjacent=False, src="bf16",
                cache="bf16", page=16, far=4093),
        # a decode batch with fp32 activations, far positions on three axes, a quarter of each head rotated, padded rows
        _append("append 256 sequences", T=256, seqs=256, n_kv=2, group=8, D=256, rd=64, axes=3, adjacent=False,
                src="f32", cache="f16", page=64, far=1000003),
        # prompts of several sequences entering the cache at once
        _append("append prompts", T=16384, seqs=11, n_kv=8, group=4, D=128, rd=128, axes=1, adjacent=True, src="bf16",
                cache="bf16", page=32, far=32768),
        # one sequence, some thousand tokens: little work for many multiprocessors
        _attn("attend 1 sequence", B=1, prefix=0, longest=4093, even=True, n_kv=8, group=4, D=128, cache="bf16", page=16),
        # a ragged decode batch without a common prefix, lengths from none to thousands
        _attn("attend ragged 61", B=61, prefix=0, longest=8192, even=False, n_kv=4, group=8, D=128, cache="f16", page=32),
        # a batch behind one system prompt, short answers so far
        _attn("attend shared 32", B=32, prefix=8191, longest=400, even=True, n_kv=8, group=4, D=128, cache="bf16", page=16),
        # many answers on one long document: the prefix is a matrix product
        _attn("attend shared 128", B=128, prefix=32768, longest=1024, even=True, n_kv=8, group=4, D=128, cache="bf16",
              page=64),
        # two very long sequences, wide heads, many queries a key head
        _attn("attend long 2", B=2, prefix=100, longest=131071, even=True, n_kv=2, group=16, D=256, cache="f16", page=128),
        # one row, the usual filters: the latency of the row-wide reductions
        _sample("sample 1 row", B=1, V=131072, src="f32", filters="k p"),
        # a small vocabulary, min-p
        _sample("sample 8 rows", B=8, V=32000, src="f16", filters="m"),
        # top-p over the whole of an odd vocabulary
        _sample("sample 64 rows", B=64, V=100003, src="bf16", filters="p"),
        # a large batch in which every row has its own settings, greedy rows and masked tokens among them
        _sample("sample 256 rows", B=256, V=200000, src="f32", filters="mixed"),
    ]


def _append(name, **c):
    return {"name": name, "op": "append", **c}


def _attn(name, **c):
    return {"name": name, "op": "attend", **c}


def _sample(name, **c):
    return {"name": name, "op": "sample", **c}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "sample"])
    while True:
        if op == "append":
            T = _log(rng, 1, 16384)
            D = rng.choice([64, 128, 256])
            c = dict(T=T, seqs=T if rng.random() < 0.4 else min(T, _log(rng, 1, 64)), n_kv=rng.choice([1, 2, 4, 8]),
                     group=rng.choice([1, 2, 3, 4, 7, 8]), D=D, rd=rng.choice([D, D, D // 2, D // 4]),
                     axes=rng.choice([1, 1, 2, 3]), adjacent=rng.random() < 0.5, src=rng.choice(["f32", "bf16", "f16"]),
                     cache=rng.choice(["bf16", "f16"]), page=rng.choice([8, 16, 24, 32, 64, 128]), far=_log(rng, 1, 1000003))
        elif op == "attend":
            c = dict(B=_log(rng, 1, 128), prefix=rng.choice([0, 1]) * _log(rng, 1, 32768), longest=_log(rng, 1, 131071),
                     even=rng.random() < 0.5, n_kv=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 4, 5, 8, 16]),
                     D=rng.choice([64, 128, 256]), cache=rng.choice(["bf16", "f16"]), page=rng.choice([8, 16, 24, 32, 64, 128]))
        else:
            c = dict(B=_log(rng, 1, 256), V=_log(rng, 1000, 200000), src=rng.choice(["f32", "bf16", "f16"]),
                     filters=rng.choice(["k p", "m", "p", "mixed", "k", "none"]))
        c["op"] = op
        w = work(c)
        most = {"append": (460e6, 1e12), "attend": (560e6, 72e9), "sample": (206e6, 1e12)}[op]
        if w["bytes"] <= most[0] and w["flops"] <= most[1]:
            return c


def _lengths(c):
    """The lengths of the rows' own keys: the same ones for every seed, which orders them."""
    B, m = c["B"], c["longest"]
    n = [max(1, m * (i + 1) // B) if c["even"] else int(m ** ((i + 1) / B)) for i in range(B)]
    n[-1] = m
    if B >= 8:
        n[0] = 0
    return n


def work(c):
    if c["op"] == "append":
        n_q = c["n_kv"] * c["group"]
        el = c["T"] * (n_q + 2 * c["n_kv"]) * c["D"]
        return {"bytes": el * (_SIZE[c["src"]] + 2) + 4 * c["T"] * (2 + c["axes"]),
                "flops": 3 * c["T"] * (n_q + c["n_kv"]) * c["rd"]}
    if c["op"] == "attend":
        own_keys, n_q = sum(_lengths(c)), c["n_kv"] * c["group"]
        return {"bytes": 2 * 2 * c["n_kv"] * c["D"] * (c["prefix"] + own_keys) + 2 * 2 * c["B"] * n_q * c["D"],
                "flops": 4 * c["D"] * n_q * (c["B"] * c["prefix"] + own_keys)}
    return {"bytes": c["B"] * (c["V"] * _SIZE[c["src"]] + 28), "flops": 4 * c["B"] * c["V"]}


# --------------------------------------------------------------------- inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[c["op"]](c, g, seed)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _prepare_append(c, g, seed):
    T, S, D, page, n_kv = c["T"], c["seqs"], c["D"], c["page"], c["n_kv"]
    n_q = n_kv * c["group"]
    rng = np.random.RandomState(seed % (1 << 31))
    per = [T // S + (i < T % S) for i in range(S)]
    start = rng.randint(0, 2 * page + 1, S)  # what the sequences have in the cache already
    pages = (int(start.max()) + max(per) + page - 1) // page
    table = torch.randperm(S * pages, generator=g, device="cuda").to(torch.int32).reshape(S, pages)
    seq = np.repeat(np.arange(S), per).astype(np.int32)
    kv_pos = (np.concatenate([np.arange(n) for n in per]) + start[seq]).astype(np.int32)
    pos = kv_pos[None, :] + rng.randint(0, c["far"] + 1, (c["axes"], 1))
    pos = pos + (rng.randint(0, 64, (c["axes"], T)) if c["axes"] > 1 else 0)
    if T >= 64:
        kv_pos[rng.randint(0, T, 3)] = -1  # padded rows
    src, cache = _T[c["src"]], _T[c["cache"]]
    qkv = _randn(g, T, (n_q + 2 * n_kv) * D, dtype=src)  # as one projection writes them
    half = c["rd"] // 2
    s = {
        "c": c,
        "q": qkv[:, :n_q * D].unflatten(1, (n_q, D)),
        "k": qkv[:, n_q * D:(n_q + n_kv) * D].unflatten(1, (n_kv, D)),
        "v": qkv[:, (n_q + n_kv) * D:].unflatten(1, (n_kv, D)),
        "k_pages": _randn(g, S * pages, n_kv, page, D, dtype=cache),
        "v_pages": _randn(g, S * pages, n_kv, page, D, dtype=cache),
        "q_out": torch.zeros((T, n_q, D), dtype=cache, device="cuda"),
        "table": table,
        "seq": torch.from_numpy(seq).cuda(),
        "kv_pos": torch.from_numpy(kv_pos).cuda(),
        "pos": torch.from_numpy(pos.astype(np.int32)).cuda(),
        "inv_freq": (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).cuda(),
        "axis": [i % c["axes"] for i in range(half)],
    }
    s["pair_axis"] = torch.tensor(s["axis"], device="cuda")
    if own:
        import quantized_expert_matvec_b200 as qx
        s["cache"] = qx.KVCache(s["k_pages"], s["v_pages"])
        s["rope"] = qx.Rope(s["inv_freq"], s["axis"], c["adjacent"])
        s["ws"] = qx.attn_workspace(s["cache"], n_q, 1)
    return s


def _prepare_attend(c, g, seed):
    B, P, D, page, n_kv = c["B"], c["prefix"], c["D"], c["page"], c["n_kv"]
    n_q = n_kv * c["group"]
    lens = np.array(_lengths(c), dtype=np.int32)
    np.random.RandomState(seed % (1 << 31)).shuffle(lens)
    used = (lens + page - 1) // page
    n_prefix = (P + page - 1) // page
    n_pages = int(used.sum()) + n_prefix + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(1, int(used.max()))), dtype=torch.int32)
    at = n_prefix + np.concatenate([[0], np.cumsum(used)[:-1]])
    slot = np.arange(table.shape[1])[None, :] + at[:, None]
    filled = torch.from_numpy(np.arange(table.shape[1])[None, :] < used[:, None]).cuda()
    table = torch.where(filled, order[torch.from_numpy(np.minimum(slot, n_pages - 1)).cuda()], 0).to(torch.int32)
    cache = _T[c["cache"]]
    s = {
        "c": c,
        "q": _randn(g, B, n_q, D, dtype=cache),
        "k_pages": _randn(g, n_pages, n_kv, page, D, dtype=cache),
        "v_pages": _randn(g, n_pages, n_kv, page, D, dtype=cache),
        "out": torch.zeros((B, n_q, D), dtype=cache, device="cuda"),
        "lse": torch.zeros((B, n_q), dtype=torch.float32, device="cuda"),
        "prefix_pages": order[:n_prefix].contiguous(),
        "table": table,
        "kv_len": torch.from_numpy(lens).cuda(),
        "scale": 1.7 / math.sqrt(D),
    }
    if own:
        import quantized_expert_matvec_b200 as qx
        s["cache"] = qx.KVCache(s["k_pages"], s["v_pages"])
        s["ws"] = qx.attn_workspace(s["cache"], n_q, B)
    return s


def _prepare_sample(c, g, seed):
    B, V = c["B"], c["V"]
    x = 2.0 * _randn(g, B, V)
    # the few tokens that a model thinks likely
    likely = torch.randint(0, V, (B, 40), generator=g, device="cuda")
    x.scatter_add_(1, likely, 4.0 + 6.0 * torch.rand((B, 40), generator=g, device="cuda"))
    s = {"c": c, "u": torch.rand(B, generator=g, device="cuda"), "temperature": None, "top_k": None, "top_p": None,
         "min_p": None}
    if c["filters"] == "mixed":
        kind = torch.arange(B, device="cuda")
        ban = torch.rand((B, V), generator=g, device="cuda") < 0.3  # tokens that a grammar forbids
        x = torch.where(ban & (kind % 5 == 0)[:, None], -math.inf, x)
        x = torch.where(ban & (kind % 5 == 1)[:, None], torch.finfo(_T[c["src"]]).min, x)
        if B >= 8:
            x[B // 2] = -math.inf  # a row that has nothing left
        s["temperature"] = torch.where(kind % 7 == 3, 0.0, 0.3 + 1.2 * torch.rand(B, generator=g, device="cuda"))
        s["top_k"] = torch.where(kind % 3 == 0, torch.randint(1, 1000, (B,), generator=g, device="cuda"), 0).to(torch.int32)
        s["top_p"] = torch.where(kind % 2 == 0, 0.5 + 0.5 * torch.rand(B, generator=g, device="cuda"), 1.0)
        s["min_p"] = torch.where(kind % 4 == 1, 0.1 * torch.rand(B, generator=g, device="cuda"), 0.0)
    else:
        s["temperature"] = torch.full((B,), 0.8, device="cuda")
        if "k" in c["filters"]:
            s["top_k"] = torch.full((B,), 50, dtype=torch.int32, device="cuda")
        if "p" in c["filters"]:
            s["top_p"] = torch.full((B,), 0.95, device="cuda")
        if "m" in c["filters"]:
            s["min_p"] = torch.full((B,), 0.05, device="cuda")
    s["logits"] = x.to(_T[c["src"]])
    s["token"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.zeros(B, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"append": _run_append, "attend": _run_attend, "sample": _run_sample}[s["c"]["op"]](s)


def _rotate(x, cos, sin, rd, adjacent):
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if adjacent else (x[..., :rd // 2], x[..., rd // 2:rd])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], dim=-1).flatten(-2) if adjacent else torch.cat([a, b], dim=-1)
    return torch.cat([turned, x[..., rd:]], dim=-1)


def _run_append(s):
    if own:
        import quantized_expert_matvec_b200 as qx
        qx.attn_kv_append(s["cache"], s["q"], s["k"], s["v"], s["table"], s["kv_pos"], s["q_out"], rope=s["rope"],
                          pos=s["pos"], seq=s["seq"], ws=s["ws"])
        return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}
    c = s["c"]
    t = (s["kv_pos"] >= 0).nonzero().squeeze(1)
    at, page = s["kv_pos"][t].long(), c["page"]
    angle = s["pos"][s["pair_axis"]].t()[t].double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    dtype = s["q_out"].dtype
    s["q_out"][t] = _rotate(s["q"][t].float(), cos, sin, c["rd"], c["adjacent"]).to(dtype)
    where = s["table"][s["seq"][t].long(), at // page].long()
    s["k_pages"][where, :, at % page] = _rotate(s["k"][t].float(), cos, sin, c["rd"], c["adjacent"]).to(dtype)
    s["v_pages"][where, :, at % page] = s["v"][t].to(dtype)
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _run_attend(s):
    c = s["c"]
    if own:
        import quantized_expert_matvec_b200 as qx
        qx.attn_decode_step(s["cache"], s["q"], s["out"], s["table"], s["kv_len"], prefix_pages=s["prefix_pages"],
                            prefix_len=c["prefix"], scale=s["scale"], lse=s["lse"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, P, D, n_kv, G = c["B"], c["prefix"], c["D"], c["n_kv"], c["group"]
    q = s["q"].float().view(B, n_kv, G, D) * s["scale"]
    kp, vp = (s[n][s["prefix_pages"].long()].transpose(0, 1).reshape(n_kv, -1, D)[:, :P].float()
              for n in ("k_pages", "v_pages"))
    ko, vo = (s[n][s["table"].long()].transpose(1, 2).reshape(B, n_kv, -1, D).float() for n in ("k_pages", "v_pages"))
    past = torch.arange(ko.shape[2], device="cuda")[None, :] >= s["kv_len"][:, None]
    sp = torch.matmul(q.transpose(0, 1).reshape(n_kv, B * G, D), kp.transpose(1, 2))
    sp = sp.view(n_kv, B, G, P).transpose(0, 1)
    so = torch.matmul(q, ko.transpose(2, 3)).masked_fill(past[:, None, None, :], -math.inf)
    m = torch.cat([sp, so], dim=-1).amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    wp, wo = torch.exp(sp - m), torch.exp(so - m)
    total = wp.sum(-1, keepdim=True) + wo.sum(-1, keepdim=True)
    o = torch.matmul(wp.transpose(0, 1).reshape(n_kv, B * G, P), vp).view(n_kv, B, G, D).transpose(0, 1)
    o = o + torch.matmul(wo, vo)
    o = torch.where(total > 0, o / total, 0.0)
    return {"out": o.reshape(B, n_kv * G, D).to(s["q"].dtype), "lse": (m + torch.log(total)).reshape(B, n_kv * G)}


def _run_sample(s):
    if own:
        import quantized_expert_matvec_b200 as qx
        qx.token_sample(s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                        top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
        return {"token": s["token"], "logprob": s["logprob"]}
    x = s["logits"].double()
    B, V = x.shape
    best = x.amax(1, keepdim=True)
    greedy = (s["temperature"] <= 0.0)[:, None]
    t = torch.where(greedy, 1.0, s["temperature"].double()[:, None])
    w = torch.where(x == best, 1.0, torch.exp((x - best) / t))  # a logit of the row's maximum weighs 1, an infinite one too
    w = torch.where(x == -math.inf, 0.0, w)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")[None, :]
    if s["top_k"] is not None:
        ws = torch.where((s["top_k"][:, None] > 0) & (rank >= s["top_k"][:, None]), 0.0, ws)
    ws = torch.where(greedy & (rank >= 1), 0.0, ws)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = ws.cumsum(1) - ws
        ws = torch.where((p < 1.0) & (before >= p * ws.sum(1, keepdim=True)) & (rank >= 1), 0.0, ws)
    if s["min_p"] is not None:
        ws = torch.where(ws < s["min_p"].double()[:, None], 0.0, ws)
    w = torch.zeros_like(w).scatter_(1, order, ws)
    cdf = w.cumsum(1)
    total = cdf[:, -1:]
    token = (cdf > s["u"].double()[:, None] * total).int().argmax(1)
    logprob = torch.log(w.gather(1, token[:, None]) / total).squeeze(1)
    none = best.squeeze(1) == -math.inf
    return {"token": torch.where(none, -1, token).to(torch.int32),
            "logprob": torch.where(none, -math.inf, logprob).float()}


# -------------------------------------------------------------- in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[c["op"]](s)


def _exact_append(s):
    c = s["c"]
    rd, half, page = c["rd"], c["rd"] // 2, c["page"]
    rows = [i for i, p in enumerate(s["kv_pos"].tolist()) if p >= 0]
    i = torch.tensor(rows, device="cuda")
    phase = torch.polar(torch.ones((len(rows), half), dtype=torch.float64, device="cuda"),
                        s["inv_freq"].double()[None, :] * s["pos"].double()[s["pair_axis"]][:, i].t())
    out = {}
    for n in ("q", "k"):
        x = s[n][i].double()
        if c["adjacent"]:
            z = torch.view_as_complex(x[..., :rd].contiguous().unflatten(-1, (half, 2)))
            x[..., :rd] = torch.view_as_real(z * phase[:, None, :]).flatten(-2)
        else:
            z = torch.complex(x[..., :half].contiguous(), x[..., half:rd].contiguous()) * phase[:, None, :]
            x[..., :half], x[..., half:rd] = z.real, z.imag
        out[n] = x
    q = s["q_out"].double()
    q[i] = out["q"]
    p = s["kv_pos"][i].long()
    dst = s["table"].long()[s["seq"][i].long(), torch.div(p, page, rounding_mode="floor")]
    off = torch.remainder(p, page)
    k, v = s["k_pages"].double(), s["v_pages"].double()
    k[dst, :, off] = out["k"]
    v[dst, :, off] = s["v"][i].double()
    return {"q": q, "k": k, "v": v}


def _exact_attend(s):
    c = s["c"]
    B, P, D, n_kv, G, page = c["B"], c["prefix"], c["D"], c["n_kv"], c["group"], c["page"]
    out = torch.zeros((B, n_kv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, n_kv * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["kv_len"].tolist()):
        pages = torch.cat([s["prefix_pages"], s["table"][b, :(n + page - 1) // page]]).long()
        n_prefix = len(s["prefix_pages"]) * page
        keep = torch.cat([torch.arange(P), n_prefix + torch.arange(n)]).cuda()
        if not len(keep):
            continue
        for h in range(n_kv):
            k = s["k_pages"][pages, h].double().reshape(-1, D)[keep]
            v = s["v_pages"][pages, h].double().reshape(-1, D)[keep]
            x = s["scale"] * (s["q"][b, h * G:(h + 1) * G].double() @ k.t())
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
            out[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def _exact_sample(s):
    x = s["logits"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    B, V = x.shape
    get = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p")}
    token, logprob = np.full(B, -1, np.int32), np.full(B, -np.inf)
    for b in range(B):
        if x[b].max() == -np.inf:
            continue
        by_size = np.argsort(-x[b], kind="stable")
        t = get["temperature"][b]
        if t <= 0:
            token[b], logprob[b] = by_size[0], 0.0
            continue
        k = 0 if get["top_k"] is None else int(get["top_k"][b])
        by_size = by_size[:k] if k > 0 else by_size
        e = np.exp((x[b][by_size] - x[b][by_size[0]]) / t)
        if get["top_p"] is not None and get["top_p"][b] < 1:
            mass = np.cumsum(e)
            n = 1 + int(np.searchsorted(mass, get["top_p"][b] * mass[-1], side="left"))
            by_size, e = by_size[:n], e[:n]
        if get["min_p"] is not None:
            n = int((e >= get["min_p"][b]).sum())
            by_size, e = by_size[:n], e[:n]
        rise = np.argsort(by_size)
        mass = np.cumsum(e[rise])
        at = min(int(np.searchsorted(mass, u[b] * mass[-1], side="right")), len(rise) - 1)
        token[b] = by_size[rise[at]]
        logprob[b] = math.log(e[rise[at]] / mass[-1])
    return {"token": torch.from_numpy(token), "logprob": torch.from_numpy(logprob)}
