"""Cases, inputs and plain forms of the operators around the MoE block of a verify step.

Three operators of one verify step over a drafted block of N tokens per sequence:

* ``block_kv_append``  - head norms of queries and keys, their position rotation, and the
  append of the block's keys and values to a paged cache, from the packed projection;
* ``block_attention``  - the block's attention over that paged cache (one new token to a
  few dozen per sequence, grouped query heads, optional sliding window);
* ``block_sample``     - probabilities and tokens from the step's logits under temperature,
  top-k, top-p and min-p, drawn with given uniforms; its probabilities are the rows that
  ``block_accept_rejection`` reads.

``own`` chooses between the library's kernels and the plain forms below (elementary torch
operations in float32; float64 and int64 where a sampled token depends on it).
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------- cases --

# Head layouts (query heads, key/value heads): grouped 8 and 4 to a head, odd groups,
# one key/value head for all, one for each.
HEADS = [(64, 8), (32, 4), (32, 8), (16, 16), (8, 1), (40, 8), (12, 2), (14, 2)]


def listed():
    return [
        # the next token of one sequence: launch latency is all there is
        _append("append_one", S=1, N=1, Hq=64, Hkv=8, D=128, rot=128, page=16, top=1000),
        # a serving batch of 8-token blocks, half of each head rotated, in neighbouring
        # pairs, two slots of the batch empty; odd page size
        _append("append_serving", S=16, N=8, Hq=40, Hkv=8, D=128, rot=64, page=24, top=2000,
                interleaved=True, idle=2),
        # the largest verify batch: 33 target rows (32 drafts and the bonus row)
        _append("append_large", S=128, N=33, Hq=64, Hkv=8, D=128, rot=128, page=64, top=700),
        # one token after a short prompt: latency of split and join
        _attention("attn_one_short", S=1, N=1, Hq=64, Hkv=8, D=128, page=16, low=777, top=777),
        # one token after 128K tokens: a single sequence has to fill the GPU
        _attention("attn_one_long", S=1, N=1, Hq=32, Hkv=4, D=128, page=16, low=131000, top=131000),
        # an 8-token block of one sequence over 32K tokens, heads of 256
        _attention("attn_block8", S=1, N=8, Hq=12, Hkv=2, D=256, page=64, low=32777, top=32777),
        # a serving batch of 8-token blocks with uneven lengths, two slots empty
        _attention("attn_serving", S=16, N=8, Hq=64, Hkv=8, D=128, page=32, low=1, top=30000, idle=2),
        # 64 sequences x 16-token blocks: 128 query rows to each key/value head
        _attention("attn_block16", S=64, N=16, Hq=32, Hkv=4, D=128, page=64, low=500, top=9000),
        # a drafter's sliding window of 128 over long sequences, heads of 64
        _attention("attn_window", S=64, N=8, Hq=16, Hkv=16, D=64, page=16, low=100, top=20000,
                   window=128),
        # next token of one sequence under every filter, as a chat sampler sets them
        _sample("sample_one", S=1, K=1, V=32000, mode="all"),
        # a serving batch: 8 rows a sequence, filters differ from sequence to sequence,
        # bf16-valued logits (many ties), probabilities and tokens
        _sample("sample_serving", S=16, K=8, V=152064, mode="mixed", coarse=True, probs=True),
        # 64 x 16 drafter rows at a temperature alone: drafts and the q rows of rejection sampling
        _sample("sample_drafts", S=64, K=16, V=32000, mode="temperature", probs=True),
    ]


def _append(name, S, N, Hq, Hkv, D, rot, page, top, norm=True, interleaved=False, idle=0):
    return {"name": name, "op": "append", "S": S, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "page": page, "top": top, "norm": norm, "interleaved": interleaved, "idle": idle}


def _attention(name, S, N, Hq, Hkv, D, page, low, top, window=0, idle=0):
    return {"name": name, "op": "attention", "S": S, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "low": low, "top": top, "window": window, "idle": idle}


def _sample(name, S, K, V, mode, coarse=False, probs=False, masked=False):
    return {"name": name, "op": "sample", "S": S, "K": K, "V": V, "mode": mode, "coarse": coarse,
            "probs": probs, "masked": masked}


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "sample", "sample"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([8, 16, 16, 24, 32, 64, 100, 128])
    if op == "append":
        S, N = _log(rng, 1, 128), _log(rng, 1, 33)
        while S * N * (Hq + 2 * Hkv) * D > 128 * 33 * 80 * 128:
            S = max(1, S // 2)
        c = _append("", S, N, Hq, Hkv, D, rng.choice([D, D, D // 2, 32, 0]), page, _log(rng, 40, 1000),
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.4,
                    idle=rng.choice([0, 0, S // 4]))
    elif op == "attention":
        S, N = _log(rng, 1, 64), _log(rng, 1, 33)
        window = rng.choice([0, 0, 0, 128, 1000])
        top = _log(rng, 1, 131072)
        # no more bytes and products than the largest listed cases
        while S * top * Hkv * D > 30000 * 16 * 8 * 128 // 2 or S * top * N * Hq * D > 64 * 4750 * 16 * 32 * 128:
            S, top = max(1, S // 2), max(1, top * 3 // 4)
        c = _attention("", S, N, Hq, Hkv, D, page, _log(rng, 1, top), top, window=window,
                       idle=rng.choice([0, 0, S // 4]))
    else:
        V = _log(rng, 1000, 152064)
        S, K = _log(rng, 1, 64), _log(rng, 1, 17)
        while S * K * V > 16 * 8 * 152064:
            S, K = max(1, S // 2), max(1, K * 3 // 4)
        c = _sample("", S, K, V, rng.choice(["all", "mixed", "mixed", "temperature", "top_k", "top_p", "min_p"]),
                    coarse=rng.random() < 0.5, probs=rng.random() < 0.5, masked=rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------ inputs --

def _lengths(c, g, low, top):
    """Cache lengths, one in each of S equal parts of low .. top; the idle slots hold 0."""
    S = c["S"]
    at = (torch.randperm(S, generator=g) + torch.rand(S, generator=g, dtype=torch.float64)) / S
    n = low + (at * (top + 1 - low)).long()
    if c["idle"]:
        n[torch.randperm(c["S"], generator=g)[:c["idle"]]] = 0
    return n


def _pages(c, lens, g, pool=None):
    """A page table in which every sequence's pages lie scattered, and the pool's size."""
    need = [-(-int(n) // c["page"]) for n in lens]
    pool = pool or sum(need) + 2
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.zeros((c["S"], max(max(need), 1) + 1), dtype=torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    return table.cuda(), pool


def _normal(shape, gg, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gg, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(c, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device="cuda").manual_seed(seed + 1)
    S = c["S"]
    if c["op"] == "append":
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        top = max(N, c["top"])
        lens = _lengths(c, g, N, top)
        table, pool = _pages(c, lens, g, S * -(-top // c["page"]) + 2)
        st = {"c": c, "kv_len": lens.to(torch.int32).cuda(), "table": table,
              "active": (lens > 0).nonzero()[:, 0].cuda(),      # the slots in use
              "qkv": _normal((S, N, Hq + 2 * Hkv, D), gg, 1.5),
              "k_cache": _normal((pool, Hkv, c["page"], D), gg),
              "v_cache": _normal((pool, Hkv, c["page"], D), gg),
              "q_out": torch.zeros((S, N, Hq, D), dtype=torch.bfloat16, device="cuda"),
              "q_weight": None, "k_weight": None, "cos_sin": None}
        if c["norm"]:
            st["q_weight"] = (1 + _normal((D,), gg, 0.1, torch.float32)).to(torch.bfloat16)
            st["k_weight"] = (1 + _normal((D,), gg, 0.1, torch.float32)).to(torch.bfloat16)
        if c["rot"]:
            h = c["rot"] // 2
            f = 1e6 ** (-torch.arange(h, dtype=torch.float64, device="cuda") / h)
            a = torch.arange(int(lens.max()) + 1, dtype=torch.float64, device="cuda")[:, None] * f
            st["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        return st
    if c["op"] == "attention":
        N, Hq, Hkv, D = c["N"], c["Hq"], c["Hkv"], c["D"]
        lens = _lengths(c, g, c["low"], c["top"])
        table, pool = _pages(c, lens, g)
        st = {"c": c, "kv_len": lens.to(torch.int32).cuda(), "table": table,
              "q": _normal((S, N, Hq, D), gg, 2.0),
              "k_cache": torch.empty((pool, Hkv, c["page"], D), dtype=torch.bfloat16, device="cuda"),
              "v_cache": torch.empty((pool, Hkv, c["page"], D), dtype=torch.bfloat16, device="cuda"),
              "out": torch.zeros((S, N, Hq, D), dtype=torch.bfloat16, device="cuda")}
        st["k_cache"].normal_(generator=gg)
        st["v_cache"].normal_(generator=gg)
        return st
    K, V = c["K"], c["V"]
    logits = torch.randn((S, K, V), generator=gg, device="cuda") * 2
    # what a model is sure of: a few tokens of every row stand out
    top = torch.randint(0, V, (S, K, 4), generator=gg, device="cuda")
    logits.scatter_add_(2, top, torch.rand((S, K, 4), generator=gg, device="cuda") * 12)
    if c["coarse"]:                     # a bf16 output layer's logits, widened: many are equal
        logits = logits.to(torch.bfloat16).float()
    if c["masked"]:                     # a grammar's mask: most tokens are not allowed
        logits.masked_fill_(torch.rand((S, K, V), generator=gg, device="cuda") < 0.9, -math.inf)
    pick = lambda values: torch.tensor(values)[torch.randint(0, len(values), (S,), generator=g)]
    on = lambda *modes: c["mode"] in modes + ("mixed", "all")
    mixed = c["mode"] != "all"
    st = {"c": c, "logits": logits,
          "u": torch.randint(0, 1 << 24, (S, K), generator=gg, device="cuda").float() * 2.0 ** -24,
          "temperature": None, "top_k": None, "top_p": None, "min_p": None}
    if on("temperature"):
        st["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.3] if mixed else [0.7, 0.9]).float().cuda()
    if on("top_k"):
        st["top_k"] = pick([0, 1, 20, 50, 1000] if mixed else [40, 64]).to(torch.int32).cuda()
    if on("top_p"):
        st["top_p"] = pick([1.0, 0.95, 0.9, 0.5] if mixed else [0.9, 0.95]).float().cuda()
    if on("min_p"):
        st["min_p"] = pick([0.0, 0.0, 0.02, 0.1] if mixed else [0.01, 0.02]).float().cuda()
    return st


# -------------------------------------------------------------------- one pass --

def run(st):
    c = st["c"]
    if own:
        import mxfp4_moe_block_b200 as mm
        if c["op"] == "append":
            mm.block_kv_append(st["qkv"], st["kv_len"], st["table"], st["k_cache"], st["v_cache"],
                               cos_sin=st["cos_sin"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                               norm=c["norm"], eps=1e-6, interleaved=c["interleaved"], q_out=st["q_out"])
            return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        if c["op"] == "attention":
            return mm.block_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"],
                                      window=c["window"], out=st["out"])
        token, probs = mm.block_sample(st["logits"], st["u"], temperature=st["temperature"],
                                       top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"],
                                       with_probs=c["probs"])
        return {"token": token, "probs": probs} if c["probs"] else {"token": token}
    return {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}[c["op"]](st)


def _plain_append(st):
    c = st["c"]
    N, Hq, Hkv, D, rot = c["N"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    a = st["active"]
    x = st["qkv"][a]
    pos = (st["kv_len"][a].long() - N)[:, None] + torch.arange(N, device="cuda")
    q, k, v = x[:, :, :Hq].float(), x[:, :, Hq:Hq + Hkv].float(), x[:, :, Hq + Hkv:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * st["q_weight"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * st["k_weight"].float()
    if rot:
        cs = st["cos_sin"][pos][:, :, None]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        q, k = (_plain_rotate(t, cos, sin, rot, c["interleaved"]) for t in (q, k))
    st["q_out"][a] = q.to(torch.bfloat16)
    page = st["table"][a].long().gather(1, pos // c["page"])
    st["k_cache"][page, :, pos % c["page"]] = k.to(torch.bfloat16)
    st["v_cache"][page, :, pos % c["page"]] = v
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_rotate(t, cos, sin, rot, interleaved):
    if interleaved:
        x, y = t[..., 0:rot:2], t[..., 1:rot:2]
        r = torch.stack([x * cos - y * sin, x * sin + y * cos], -1).flatten(-2)
    else:
        x, y = t[..., :rot // 2], t[..., rot // 2:rot]
        r = torch.cat([x * cos - y * sin, x * sin + y * cos], -1)
    return torch.cat([r, t[..., rot:]], -1)


def _plain_attention(st):
    c = st["c"]
    S, N, Hq, Hkv, D, page, W = c["S"], c["N"], c["Hq"], c["Hkv"], c["D"], c["page"], c["window"]
    G, table, n = Hq // Hkv, st["table"], st["kv_len"].long()[:, None]
    # the pages that a block's window can touch, or all of them
    cols = torch.arange(min(table.shape[1], (W + N) // page + 2) if W else table.shape[1], device="cuda")
    cols = cols + ((n - N - W + 1).clamp(min=0) // page if W else 0 * n)
    p = table.gather(1, cols.clamp(max=table.shape[1] - 1)).long()
    key = (cols[:, :, None] * page + torch.arange(page, device="cuda")).view(S, 1, -1)
    pos = (n - N + torch.arange(N, device="cuda"))[:, :, None]
    see = key <= pos                                                     # [S, N, keys]
    if W:
        see = see & (key > pos - W)
    k = st["k_cache"][p].transpose(1, 2).reshape(S, Hkv, -1, D).float()
    q = st["q"].view(S, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, N * G, D).float()
    z = torch.matmul(q, k.transpose(2, 3)).view(S, Hkv, N, G, -1) * D ** -0.5
    del k
    z = z.masked_fill(~see[:, None, :, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    e = e / e.sum(-1, keepdim=True).clamp(min=1e-30)                     # a row that sees no key: 0
    v = st["v_cache"][p].transpose(1, 2).reshape(S, Hkv, -1, D).float()
    o = torch.matmul(e.view(S, Hkv, N * G, -1), v).view(S, Hkv, N, G, D)
    st["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(S, N, Hq, D))
    return st["out"]


def _plain_sample(st):
    c = st["c"]
    S, K, V = c["S"], c["K"], c["V"]
    row = lambda t: t.repeat_interleave(K)[:, None]        # a sequence's setting, for its K rows
    l = st["logits"].view(S * K, V)
    top = l.amax(1, keepdim=True)
    z = l.double() - top.double()
    cold = None
    if st["temperature"] is not None:
        t = row(st["temperature"]).double()
        cold = t <= 0
        z = z / torch.where(cold, 1.0, t)
    w = torch.exp(z)
    mass = torch.floor(w * 2.0 ** 40).long()
    keep = None
    if any(st[k] is not None for k in ("temperature", "top_k", "top_p", "min_p")):
        order = torch.sort(l, dim=1, descending=True, stable=True).indices
        m = mass.gather(1, order)
        rank = torch.arange(V, device="cuda")[None]
        stay = torch.ones_like(m, dtype=torch.bool)
        if st["top_k"] is not None:
            k = row(st["top_k"])
            stay = (rank < k) | (k <= 0)
        if st["top_p"] is not None:
            p = row(st["top_p"]).double()
            m = torch.where(stay, m, 0)
            run_ = m.cumsum(1)
            bar = torch.ceil(p * run_[:, -1:].double()).long()
            stay = stay & ((run_ - m < bar) | (p >= 1))
        if st["min_p"] is not None:
            low = torch.floor(row(st["min_p"]).double() * 2.0 ** 40).long()
            stay = stay & ((m >= low) | (rank == 0))
        if cold is not None:
            stay = torch.where(cold, rank == 0, stay)
        keep = torch.zeros_like(stay).scatter_(1, order, stay)
        mass = torch.where(keep, mass, 0)
    run_ = mass.cumsum(1)
    U = (st["u"].view(-1, 1).double() * 2.0 ** 24).long()
    total = run_[:, -1:]
    m = (total >> 24) * U + (((total & 0xffffff) * U) >> 24)
    token = (run_ <= m).sum(1).to(torch.int32).view(S, K)
    if not c["probs"]:
        return {"token": token}
    if keep is not None:
        w = torch.where(keep, w, 0.0)
    return {"token": token, "probs": (w / w.sum(1, keepdim=True)).float().view(S, K, V)}


# --------------------------------------------------------------- floors of a pass --

def _mean_length(c):
    return (c["S"] - c["idle"]) * (c["low"] + c["top"]) / 2


def work(c):
    S = c["S"]
    if c["op"] == "append":
        tokens = (S - c["idle"]) * c["N"]
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": tokens * (2 * heads * c["D"] * 2 + c["rot"] * 4),
                "flops": tokens * (c["Hq"] + c["Hkv"]) * (c["D"] * (4 if c["norm"] else 0) + c["rot"] * 3)}
    if c["op"] == "attention":
        keys = _mean_length(c)
        if c["window"]:
            keys = min(keys, (S - c["idle"]) * (c["window"] + c["N"]))
        return {"bytes": keys * c["Hkv"] * c["D"] * 4 + S * c["N"] * c["Hq"] * c["D"] * 4,
                "flops": keys * c["N"] * c["Hq"] * c["D"] * 4}
    n = S * c["K"] * c["V"]
    return {"bytes": n * (8 if c["probs"] else 4), "flops": n * 20}


# ---------------------------------------------------------------- the definition --

def exact(c, seed):
    st = prepare(c, seed)
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[c["op"]](st)


def _exact_append(st):
    """Every head as complex numbers (the rotation is a product) in float64."""
    c = st["c"]
    N, Hq, Hkv, D, rot, page = c["N"], c["Hq"], c["Hkv"], c["D"], c["rot"], c["page"]
    out = {"q": st["q_out"].double(), "k_cache": st["k_cache"].double(), "v_cache": st["v_cache"].double()}
    for s in range(c["S"]):
        n = int(st["kv_len"][s])
        if n == 0:
            continue
        x = st["qkv"][s].double()
        heads = []
        for a, b, w in ((0, Hq, st["q_weight"]), (Hq, Hq + Hkv, st["k_weight"])):
            t = x[:, a:b]
            if c["norm"]:
                t = t / (t.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            if rot:
                cs = st["cos_sin"][n - N:n].double()
                turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
                if c["interleaved"]:
                    even, odd = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
                else:
                    even, odd = torch.arange(rot // 2), torch.arange(rot // 2, rot)
                y = torch.complex(t[..., even], t[..., odd]) * turn
                t = t.clone()
                t[..., even], t[..., odd] = y.real, y.imag
            heads.append(t)
        out["q"][s] = heads[0]
        for i in range(N):
            p, at = divmod(n - N + i, page)
            p = int(st["table"][s, p])
            out["k_cache"][p, :, at] = heads[1][i]
            out["v_cache"][p, :, at] = x[i, Hq + Hkv:]
    return out


def _exact_attention(st):
    """Token by token of the block: softmax over the keys it sees, in float64."""
    c = st["c"]
    N, Hq, Hkv, D, page, W = c["N"], c["Hq"], c["Hkv"], c["D"], c["page"], c["window"]
    out = torch.zeros((c["S"], N, Hq, D), dtype=torch.float64, device="cuda")
    for s in range(c["S"]):
        n = int(st["kv_len"][s])
        lo = max(0, n - N + 1 - W) if W else 0
        j = torch.arange(lo, n, device="cuda")
        p, at = st["table"][s].long()[j // page], j % page
        k, v = st["k_cache"][p, :, at].double(), st["v_cache"][p, :, at].double()     # [n, Hkv, D]
        for i in range(N):
            last = n - N + i
            if last < 0:
                continue
            a = max(0, last - W + 1) - lo if W else 0
            q = st["q"][s, i].double().view(Hkv, Hq // Hkv, D)
            z = torch.einsum("hgd,nhd->hgn", q, k[a:last + 1 - lo]) / math.sqrt(D)
            out[s, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), v[a:last + 1 - lo]).reshape(Hq, D)
    return out


def _exact_sample(st):
    """Row by row in numpy: the ranking's prefix that every filter lets stay, and the
    integer draw over it in token order."""
    c = st["c"]
    S, K, V = c["S"], c["K"], c["V"]
    l = st["logits"].cpu().numpy().astype(np.float64)
    u = st["u"].cpu().numpy().astype(np.float64)
    opt = {k: (None if st[k] is None else st[k].cpu().numpy()) for k in ("temperature", "top_k", "top_p", "min_p")}
    token = np.zeros((S, K), np.int32)
    probs = np.zeros((S, K, V)) if c["probs"] else None
    for s in range(S):
        t = 1.0 if opt["temperature"] is None else float(opt["temperature"][s])
        for i in range(K):
            x = l[s, i]
            if t <= 0:
                token[s, i] = int(x.argmax())
                if c["probs"]:
                    probs[s, i, token[s, i]] = 1
                continue
            w = np.exp((x - x.max()) / t)
            mass = np.floor(w * 2.0 ** 40).astype(np.int64)
            n = V
            rank = np.lexsort((np.arange(V), -x)) if any(opt[k] is not None for k in ("top_k", "top_p", "min_p")) \
                else np.arange(V)
            if opt["top_k"] is not None and 0 < opt["top_k"][s] < V:
                n = int(opt["top_k"][s])
            cum = np.cumsum(mass[rank[:n]])
            if opt["min_p"] is not None:
                m = int(np.count_nonzero(mass[rank[:n]] >= int(float(opt["min_p"][s]) * 2.0 ** 40)))
            else:
                m = n
            if opt["top_p"] is not None and opt["top_p"][s] < 1:
                bar = math.ceil(float(opt["top_p"][s]) * float(cum[-1]))
                n = min(n, int(np.searchsorted(cum, bar, side="left")) + 1)
            n = max(1, min(n, m))
            kept = np.sort(rank[:n])
            cum = np.cumsum(mass[kept])
            m = (int(cum[-1]) * int(u[s, i] * 2 ** 24)) >> 24
            token[s, i] = kept[np.searchsorted(cum, m, side="right")]
            if c["probs"]:
                probs[s, i, kept] = w[kept] / w[kept].sum()
    token = torch.from_numpy(token).cuda()
    return {"token": token, "probs": torch.from_numpy(probs).cuda()} if c["probs"] else {"token": token}
