"""The cached-serving operators: what is measured of them, and their plain forms.

Four entry points of ``sparse_attention_08_b200`` that belong to one serving
step over a paged latent cache (576-d latents, the first 512 dims the value):

* ``decode``  dsa_paged_mla_decode: attention of one new token per sequence
  over its paged latents, optionally only a sliding window and the first tokens;
* ``mass``    dsa_paged_attn_mass: the attention weight each cached entry got
  from that token, summed over the heads and added to a running total;
* ``evict``   dsa_cache_evict: the cache cut down to a budget of entries by
  that total, the first and the newest entries always kept;
* ``window``  dsa_window_mha_fwd: the prompt's attention in the MHA form (192-d
  queries and keys, 128-d values) over a sliding window and the first tokens.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is set, by the framework's calls.
"""
import math
import random

import torch

own = False

D, DV = 576, 512            # latent, value part
MHA_DQK, MHA_DV = 192, 128  # query/key and value dims of the MHA form


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the decode batch of the benchmark: 64 sequences with caches of 4096..131072 tokens
        dict(name="decode-batch64-h128", op="decode", B=64, lo=4096, hi=131072, H=128, page=64,
             window=0, sinks=0, lens=11),
        # one user with a full 128K context: the cache has to be split to fill the GPU
        dict(name="decode-one-long-h128", op="decode", B=1, lo=130949, hi=130949, H=128, page=64,
             window=0, sinks=0, lens=12),
        # the first tokens of a few short chats, few heads per GPU: latency
        dict(name="decode-short-h16", op="decode", B=3, lo=1, hi=1000, H=16, page=16, window=0,
             sinks=0, lens=13),
        # a busy server with a windowed layer, heads split over two GPUs
        dict(name="decode-window-h64", op="decode", B=48, lo=2049, hi=65536, H=64, page=32,
             window=4096, sinks=4, lens=14),
        # attention totals of a batch with long caches
        dict(name="mass-batch16-h128", op="mass", B=16, lo=4096, hi=131072, H=128, page=64,
             window=0, sinks=0, lens=15),
        # the same for short chats in a windowed layer
        dict(name="mass-short-h16", op="mass", B=5, lo=1, hi=2500, H=16, page=16, window=512,
             sinks=4, lens=16),
        # a batch of full contexts cut down to 8192 entries each
        dict(name="evict-batch8-to-8192", op="evict", B=8, lo=100000, hi=131072, page=64,
             budget=8192, sinks=4, recent=1024, lens=17),
        # one long context cut down to the selection size of the sparse attention
        dict(name="evict-one-to-2048", op="evict", B=1, lo=131072, hi=131072, page=128,
             budget=2048, sinks=4, recent=128, lens=18),
        # short chats, most of them under the budget
        dict(name="evict-short", op="evict", B=5, lo=1, hi=1500, page=16, budget=256, sinks=4,
             recent=32, lens=19),
        # the short-prefill prompt of the benchmark (L = 4096, 128 heads), windowed
        dict(name="window-prompt4096-h128", op="window", B=1, lo=4096, hi=4096, qlen=0, H=128,
             window=1024, sinks=4, lens=20),
        # chunks of 1000 new tokens against caches of up to 16384
        dict(name="window-chunk1000-h64", op="window", B=2, lo=9001, hi=16384, qlen=1000, H=64,
             window=4096, sinks=16, lens=21),
        # short prompts, few heads: latency
        dict(name="window-short-h16", op="window", B=3, lo=1, hi=300, qlen=0, H=16, window=128,
             sinks=4, lens=22),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "mass", "evict", "window"])
    c = dict(op=op, lens=rng.randrange(1 << 30))
    if op == "window":
        H = rng.choice([1, 2, 7, 16, 32, 64, 128])
        hi = _log_int(rng, 1, 4096 if H > 64 else 8192)
        # the score matrix of the plain form: B * H * L * L values
        B = _log_int(rng, 1, max(1, min(16, (1 << 31) // (H * hi * hi))))
        c.update(B=B, lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, H=H,
                 qlen=rng.choice([0, 0, 1, _log_int(rng, 1, hi)]),
                 window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 130]))
        return c
    B = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, min(131072, (16 if op == "mass" else 64) * 65536 // B))
    c.update(B=B, lo=max(1, hi // rng.choice([1, 2, 30])), hi=hi,
             page=rng.choice([16, 32, 48, 64, 128, 256]))
    if op == "evict":
        c["hi"] = hi = min(hi, (1 << 20) // B)
        c["lo"] = min(c["lo"], hi)
        budget = _log_int(rng, 1, 8192)
        sinks = min(rng.choice([0, 1, 4, 64]), budget)
        c.update(budget=budget, sinks=sinks,
                 recent=min(budget - sinks, rng.choice([0, 1, 32, 1024])))
    else:
        c.update(H=rng.choice([16, 32, 64, 128]),
                 window=rng.choice([0, 0, _log_int(rng, 1, 8192)]),
                 sinks=rng.choice([0, 1, 4, 100]))
    return c


def _lens(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _pages(n, page):
    return -(-n // page)


def _visible(n, window, sinks):
    """How many of n cached entries the newest token sees."""
    if window <= 0:
        return n
    near = min(n, window)
    return near + min(sinks, n - near)


# ---------------------------------------------------------------- inputs
def _normal(shape, g, dev, scale=1.0):
    """bf16 normal values, made in pieces so that a large cache needs no 32-bit copy."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    flat = x.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=dev).mul_(scale).to(torch.bfloat16)
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens = _lens(case)
    s = dict(case=case)
    if case["op"] == "window":
        ql = [min(case["qlen"], n) or n for n in lens]
        H = case["H"]
        s["cu_q"] = torch.tensor([0] + ql, device=dev).cumsum(0).to(torch.int32)
        s["cu_k"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        s["max_q"], s["max_k"] = max(ql), max(lens)
        s["q"] = _normal((sum(ql), H, MHA_DQK), g, dev, 2.0)
        s["k"] = _normal((sum(lens), H, MHA_DQK), g, dev)
        s["v"] = _normal((sum(lens), H, MHA_DV), g, dev)
        s["scale"] = MHA_DQK ** -0.5
        s["out"] = torch.empty((sum(ql), H, MHA_DV), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((sum(ql), H), dtype=torch.float32, device=dev)
        return s
    # a pool of pages in no order, as a server's allocator hands them out
    B, page, most = case["B"], case["page"], max(lens)
    need = [_pages(n, page) for n in lens]
    extra = [_pages(min(n, case["budget"]), page) for n in lens] if case["op"] == "evict" else [0] * B
    order = torch.randperm(sum(need) + sum(extra), generator=g, device=dev).to(torch.int32)
    s["pool"] = _normal((sum(need) + sum(extra), page, D), g, dev)
    s["table"] = _table(order, need, max(need), dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["max_len"] = most
    if case["op"] == "evict":
        s["new_table"] = _table(order[sum(need):], extra, max(extra), dev)
        # running totals: heavy-tailed, and some entries that nothing ever looked at
        m = torch.randn((B, most), generator=g, device=dev).mul_(2.0).exp_()
        s["mass"] = m.masked_fill_(torch.rand((B, most), generator=g, device=dev) < 0.1, 0.0)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["idx"] = torch.empty((B, case["budget"]), dtype=torch.int32, device=dev)
        s["new_mass"] = torch.empty((B, case["budget"]), dtype=torch.float32, device=dev)
        return s
    s["q"] = _normal((B, case["H"], D), g, dev, 2.0)
    s["scale"] = D ** -0.5
    s["lse"] = torch.empty((B, case["H"]), dtype=torch.float32, device=dev)
    if case["op"] == "decode":
        s["out"] = torch.empty((B, case["H"], DV), dtype=torch.bfloat16, device=dev)
    else:
        # the log-sum-exps that the attention call left, and the totals so far
        s["lse"] = torch.logsumexp(_scores(s), -1).clamp_min_(-1e30)
        s["mass_in"] = torch.rand((B, most), generator=g, device=dev) * 10
        s["mass"] = torch.zeros((B, most), dtype=torch.float32, device=dev)
    return s


def _table(order, need, cols, dev):
    """Block table [B, cols]: need[b] pages of row b from `order`, then zeros."""
    n = torch.tensor(need, device=dev)
    first = n.cumsum(0) - n
    j = torch.arange(cols, device=dev)
    at = (first[:, None] + j).clamp_max(order.numel() - 1)
    return torch.where(j < n[:, None], order[at], 0).to(torch.int32).contiguous()


# ---------------------------------------------------------------- one pass
def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import sparse_attention_08_b200 as dsa
    c = s["case"]
    if c["op"] == "decode":
        dsa.dsa_paged_mla_decode(s["q"], s["pool"], s["table"], s["lens"], s["max_len"],
                                 s["scale"], s["out"], s["lse"], window=c["window"],
                                 sinks=c["sinks"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        dsa.dsa_paged_attn_mass(s["q"], s["pool"], s["table"], s["lens"], s["lse"], s["max_len"],
                                s["scale"], s["mass"], mass_in=s["mass_in"], window=c["window"],
                                sinks=c["sinks"])
        return {"mass": s["mass"]}
    if c["op"] == "evict":
        dsa.dsa_cache_evict(s["pool"], s["table"], s["lens"], s["mass"], s["max_len"],
                            c["budget"], c["sinks"], c["recent"], s["new_table"], s["new_lens"],
                            s["idx"], s["new_mass"])
        return {"pool": s["pool"], "lens": s["new_lens"], "idx": s["idx"], "mass": s["new_mass"]}
    dsa.dsa_window_mha_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], c["B"], s["max_q"],
                           s["max_k"], c["window"], c["sinks"], s["scale"], s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain(s):
    return {"decode": _decode, "mass": _mass, "evict": _evict, "window": _window}[s["case"]["op"]](s)


def _latents(s):
    """The cached latents as [B, max_len, 576] in 32 bits."""
    x = s["pool"][s["table"].long()]
    return x.view(x.shape[0], -1, D)[:, :s["max_len"]].float()


def _seen(s):
    """[B, max_len]: the entries that the newest token sees."""
    c, n = s["case"], s["lens"].long()[:, None]
    j = torch.arange(s["max_len"], device=n.device)
    ok = j < n
    return ok & ((j >= n - c["window"]) | (j < c["sinks"])) if c["window"] else ok


def _scores(s, x=None):
    x = _latents(s) if x is None else x
    z = torch.matmul(s["q"].float(), x.transpose(1, 2)).mul_(s["scale"])
    return z.masked_fill_(~_seen(s)[:, None], -math.inf)


def _decode(s):
    x = _latents(s)
    z = _scores(s, x)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, x[..., :DV]) / total
    return {"out": out.to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def _mass(s):
    w = (_scores(s) - s["lse"][..., None]).exp_().sum(1)
    j = torch.arange(s["max_len"], device=w.device)
    return {"mass": torch.where(j < s["lens"][:, None], s["mass_in"] + w, s["mass"])}


def _evict(s):
    c, dev = s["case"], s["mass"].device
    n = s["lens"].long()[:, None]
    j = torch.arange(s["max_len"], device=dev)
    kept = n.clamp_max(c["budget"])
    key = s["mass"].masked_fill((j < c["sinks"]) | (j >= n - c["recent"]), math.inf)
    key = key.masked_fill(j >= n, -1.0)
    rank = key.sort(dim=1, descending=True, stable=True).indices[:, :c["budget"]]
    slot = torch.arange(rank.shape[1], device=dev)
    idx = rank.masked_fill(slot >= kept, s["max_len"]).sort(dim=1).values
    live = slot < kept
    at = idx.masked_fill(~live, 0)
    page = c["page"]
    src = s["table"].long().gather(1, at // page) * page + at % page
    dst = s["new_table"].long()[:, slot // page] * page + slot % page
    rows = s["pool"].view(-1, D)
    rows[dst[live]] = rows[src[live]]
    s["idx"].fill_(-1)
    s["idx"][:, :rank.shape[1]] = idx.masked_fill(~live, -1).to(torch.int32)
    s["new_mass"].zero_()
    s["new_mass"][:, :rank.shape[1]] = s["mass"].gather(1, at).masked_fill(~live, 0.0)
    return {"pool": s["pool"], "lens": kept.squeeze(1).to(torch.int32), "idx": s["idx"],
            "mass": s["new_mass"]}


def _padded(x, cu, most):
    """Packed rows [T, H, d] as [B, H, most, d] in 32 bits, zeros behind each sequence, and where they are real."""
    n = (cu[1:] - cu[:-1]).long()[:, None]
    j = torch.arange(most, device=x.device)
    at = (cu[:-1].long()[:, None] + j).clamp_max(x.shape[0] - 1)
    ok = j < n
    return x[at].masked_fill(~ok[..., None, None], 0).transpose(1, 2).float(), ok


def _window(s):
    c = s["case"]
    q, real = _padded(s["q"], s["cu_q"], s["max_q"])
    k, ok = _padded(s["k"], s["cu_k"], s["max_k"])
    v, _ = _padded(s["v"], s["cu_k"], s["max_k"])
    len_q, len_k = ((cu[1:] - cu[:-1]).long()[:, None, None] for cu in (s["cu_q"], s["cu_k"]))
    p = len_k - len_q + torch.arange(s["max_q"], device=q.device)[:, None]
    j = torch.arange(s["max_k"], device=q.device)
    see = ok[:, None] & (j <= p) & ((j > p - c["window"]) | (j < c["sinks"]))
    z = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~see[:, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = (torch.matmul(e, v) / total).transpose(1, 2)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2)
    return {"out": out[real].to(torch.bfloat16), "lse": lse[real]}


# ---------------------------------------------------------------- costs
def work(case):
    lens = _lens(case)
    B = case["B"]
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        pages = sum(_pages(min(n, case["budget"]), case["page"]) for n in lens)
        # the totals once; each kept latent read and written, its total and its position written
        return {"bytes": 4 * sum(lens) + kept * (2 * 2 * D + 4 + 4) + 8 * pages + 8 * B,
                "flops": sum(lens)}
    H = case["H"]
    if case["op"] == "window":
        pairs, rows, read = 0, 0, 0
        for n in lens:
            m = min(case["qlen"], n) or n
            rows += m
            pairs += sum(_visible(p + 1, case["window"], case["sinks"]) for p in range(n - m, n))
            near = min(n, m + case["window"] - 1)
            read += near + min(case["sinks"], n - near)
        return {"bytes": 2 * H * (rows * (MHA_DQK + MHA_DV) + read * (MHA_DQK + MHA_DV)) + 4 * rows * H,
                "flops": 2 * H * pairs * (MHA_DQK + MHA_DV)}
    seen = sum(_visible(n, case["window"], case["sinks"]) for n in lens)
    table = 4 * sum(_pages(n, case["page"]) for n in lens)
    if case["op"] == "decode":
        return {"bytes": 2 * D * seen + table + B * H * (2 * D + 2 * DV + 4),
                "flops": 2 * H * seen * (D + DV)}
    return {"bytes": 2 * D * seen + table + B * H * (2 * D + 4) + 8 * sum(lens),
            "flops": 2 * H * seen * D}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens = _lens(case)
    if case["op"] == "evict":
        return _exact_evict(s, lens)
    if case["op"] == "window":
        return _exact_window(s)
    out, lse, mass = [], [], s["mass"].double() if case["op"] == "mass" else None
    for b, n in enumerate(lens):
        pages = s["table"][b, :_pages(n, case["page"])].long()
        x = s["pool"][pages].reshape(-1, D)[:n]
        pos = list(range(n))
        if case["window"]:
            first = max(0, n - case["window"])
            pos = list(range(min(case["sinks"], first))) + pos[first:]
        pos = torch.tensor(pos, device=x.device)
        x = x[pos].double()
        z = x @ s["q"][b].double().T * s["scale"]               # [seen, H]
        if case["op"] == "mass":
            w = torch.exp(z - s["lse"][b].double()).sum(1)
            mass[b, :n] = s["mass_in"][b, :n].double()
            mass[b, pos] += w
            continue
        ls = torch.logsumexp(z, 0)
        out.append(torch.exp(z - ls).T @ x[:, :DV])
        lse.append(ls)
    return {"mass": mass} if case["op"] == "mass" else {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_evict(s, lens):
    c = s["case"]
    B, budget, page = c["B"], c["budget"], c["page"]
    pool = s["pool"]
    rows = pool.view(-1, D)
    idx = torch.full((B, budget), -1, dtype=torch.int64)
    mass = torch.zeros((B, budget), dtype=torch.float64)
    total = s["mass"].double().cpu()
    table, new = s["table"].cpu().long(), s["new_table"].cpu().long()
    for b, n in enumerate(lens):
        keep = list(range(n))
        if n > budget:
            mid = keep[c["sinks"]:n - c["recent"]]
            row = total[b].tolist()
            mid.sort(key=lambda i: (-row[i], i))
            room = budget - c["sinks"] - c["recent"]
            keep = sorted(keep[:c["sinks"]] + mid[:room] + keep[n - c["recent"]:])
        at = torch.tensor(keep)
        to = torch.arange(len(keep))
        idx[b, :len(keep)] = at
        mass[b, :len(keep)] = total[b, at]
        src = table[b, at // page] * page + at % page
        dst = new[b, to // page] * page + to % page
        rows[dst.to(rows.device)] = rows[src.to(rows.device)]
    return {"pool": pool, "lens": torch.tensor([min(n, budget) for n in lens]), "idx": idx,
            "mass": mass}


def _exact_window(s):
    c = s["case"]
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    outs, lses = [], []
    for b in range(c["B"]):
        q = s["q"][cq[b]:cq[b + 1]]
        k, v = s["k"][ck[b]:ck[b + 1]], s["v"][ck[b]:ck[b + 1]]
        p = torch.arange(k.shape[0] - q.shape[0], k.shape[0], device=q.device)[:, None]
        j = torch.arange(k.shape[0], device=q.device)
        hidden = (j > p) | ((p - j >= c["window"]) & (j >= c["sinks"]))
        o, ls = [], []
        for h in range(c["H"]):
            z = q[:, h].double() @ k[:, h].double().T * s["scale"]
            z[hidden] = -math.inf
            t = torch.logsumexp(z, 1)
            o.append(torch.exp(z - t[:, None]) @ v[:, h].double())
            ls.append(t)
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(ls, 1))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
