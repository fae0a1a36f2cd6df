"""The serving operators around the NVFP4 projections, as cases that can be timed and checked.

Where `own` is false, `run` computes an operator from elementary torch operations in 32 bits and
rounds once at the end; where it is true, it makes the library's call.  Four operators:

  plan    block tables and slot maps from request lengths
  append  new key and value rows into the paged cache (bf16, or e4m3 with a scale)
  attn    attention of each request's newest tokens over its paged cache
  lora    low-rank adapters of many requests beside a shared projection
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a speculative verify round of a small batch: eight new tokens each
        {"name": "plan verify 32", "op": "plan", "requests": 32, "new": "eight", "longest": 4096,
         "block": 16, "pad": 0},
        # a large mixed batch: decode tokens beside prefill chunks, idle requests among them
        {"name": "plan mixed 1024", "op": "plan", "requests": 1024, "new": "mixed",
         "longest": 16384, "block": 16, "pad": 37},
        # the same verify round's keys and values, out of the fused qkv projection's rows
        {"name": "append verify 128 bf16", "op": "append", "tokens": 128, "heads": 4, "dim": 256,
         "block": 16, "e4m3": False, "skip": False},
        # a prefill chunk into an 8-bit cache, padded rows among it
        {"name": "append chunk 8192 e4m3", "op": "append", "tokens": 8192, "heads": 4, "dim": 256,
         "block": 64, "e4m3": True, "skip": True},
        # one user, a short conversation: latency
        {"name": "decode 1 x 517", "op": "attn", "requests": 1, "longest": 517, "spread": False,
         "new": 1, "heads": 24, "kv_heads": 4, "dim": 256, "block": 16, "e4m3": False},
        # a serving batch of very different lengths, one token each
        {"name": "decode 64 ragged", "op": "attn", "requests": 64, "longest": 8192, "spread": True,
         "new": 1, "heads": 24, "kv_heads": 4, "dim": 256, "block": 16, "e4m3": False},
        # verify rounds on an 8-bit cache with another head geometry
        {"name": "verify 16 x 8 e4m3", "op": "attn", "requests": 16, "longest": 16001,
         "spread": True, "new": 8, "heads": 32, "kv_heads": 8, "dim": 128, "block": 32,
         "e4m3": True},
        # one user with a very long context: a single row of work to split over the GPU
        {"name": "decode 1 x 131072", "op": "attn", "requests": 1, "longest": 131072,
         "spread": False, "new": 1, "heads": 24, "kv_heads": 4, "dim": 256, "block": 64,
         "e4m3": False},
        # a prefill chunk in the middle of a long prompt
        {"name": "chunk 2048 over 16384", "op": "attn", "requests": 1, "longest": 16384,
         "spread": False, "new": 2048, "heads": 24, "kv_heads": 4, "dim": 256, "block": 16,
         "e4m3": False},
        # one row with one small adapter beside the input projection: latency
        {"name": "lora 1 row rank 16", "op": "lora", "rows": 1, "adapters": 4, "rank": 16,
         "mixed": False, "n": 10240, "k": 5120, "bare": False},
        # a few requests sharing adapters of different ranks beside the down projection
        {"name": "lora 37 rows mixed ranks", "op": "lora", "rows": 37, "adapters": 9, "rank": 64,
         "mixed": True, "n": 5120, "k": 17408, "bare": True},
        # the largest decode batch over many adapters
        {"name": "lora 128 rows 48 adapters", "op": "lora", "rows": 128, "adapters": 48,
         "rank": 64, "mixed": False, "n": 10240, "k": 5120, "bare": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "lora", "lora"])
    if op == "plan":
        return {"op": op, "requests": _log(rng, 1, 1024),
                "new": rng.choice(["one", "eight", "mixed"]), "longest": _log(rng, 64, 16384),
                "block": rng.choice([16, 32, 64, 128]), "pad": rng.randrange(0, 40)}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.choice([1, 2, 4]),
                "dim": rng.choice([64, 128, 256]), "block": rng.choice([16, 32, 64, 128]),
                "e4m3": rng.random() < 0.5, "skip": rng.random() < 0.5}
    if op == "lora":
        return {"op": op, "rows": _log(rng, 1, 128), "adapters": _log(rng, 1, 48),
                "rank": rng.choice([16, 32, 48, 64]), "mixed": rng.random() < 0.5,
                "n": rng.choice([1024, 5120, 6144, 10240]), "k": rng.choice([5120, 6144]),
                "bare": rng.random() < 0.5}
    kv_heads, group = rng.choice([(4, 6), (8, 4), (1, 7), (2, 8), (5, 1)])
    base = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads,
            "dim": rng.choice([64, 128, 256]), "block": rng.choice([16, 32, 64, 128]),
            "e4m3": rng.random() < 0.4}
    kind = rng.choice(["decode", "verify", "chunk"])
    if kind == "chunk":
        new = _log(rng, 16, 1024)
        requests = rng.choice([1, 1, 2, 3])
        longest = new + _log(rng, 1, 8192)
    else:
        new = 1 if kind == "decode" else rng.randrange(2, 9)
        requests = _log(rng, 1, 64)
        longest = new + _log(rng, 1, max(2, min(65536, 262144 // requests)))
    return dict(base, requests=requests, longest=longest, spread=requests > 1, new=new)


def _case_rng(case):
    """Lengths belong to the case, not to the seed: the same work for every seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _plan_sizes(case):
    rng, n = _case_rng(case), case["requests"]
    lens = [rng.randrange(0, case["longest"] + 1) for _ in range(n)]
    if case["new"] == "one":
        new = [1] * n
    elif case["new"] == "eight":
        new = [8] * n
    else:  # mostly decode, some idle, a few chunks
        new = [rng.choice([0, 1, 1, 1, 1, 1, 1, 8, 8, rng.randrange(1, 160)]) for _ in range(n)]
    return lens, new


def _attn_sizes(case):
    """(tokens in the cache, new ones among them) of each request."""
    rng, n = _case_rng(case), case["requests"]
    if not case["spread"]:
        return [case["longest"]] * n, [case["new"]] * n
    new = [case["new"] if case["new"] <= 8 else rng.randrange(1, case["new"] + 1)
           for _ in range(n)]
    new[0] = case["new"]
    lens = [rng.randrange(m, case["longest"] + 1) for m in new]
    lens[0] = case["longest"]
    return lens, new


def _lora_index(case):
    rng, m = _case_rng(case), case["rows"]
    index = [rng.randrange(case["adapters"]) for _ in range(m)]
    if case["bare"]:  # requests without an adapter
        index = [-1 if rng.random() < 0.2 else a for a in index]
        index[0] = 0
    step = 8
    ranks = [case["rank"] if not case["mixed"] else step * rng.randrange(1, case["rank"] // step + 1)
             for _ in range(case["adapters"])]
    return index, ranks


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, dtype=torch.bfloat16, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    for at in range(0, flat.numel(), 1 << 28):  # bounded fp32 temporaries
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(scale))
    return t


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(g, pages, spare, columns):
    """Random pages: a table row per request, unowned columns -1, and the pages left over."""
    total = sum(pages) + spare
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    count = _ints(pages)
    first = torch.cumsum(count, 0) - count
    col = torch.arange(columns, device="cuda")
    at = (first[:, None] + col).clamp(max=max(total - 1, 0))
    table = torch.where(col < count[:, None], perm[at], -1).to(torch.int32)
    return table, perm[sum(pages):].contiguous(), total


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "plan":
        lens, new = _plan_sizes(case)
        b = case["block"]
        columns = (max(lens) + max(new)) // b + 2
        wanted = sum(-(-(n + m) // b) - -(-n // b) for n, m in zip(lens, new))
        table, free, _ = _tables(g, [-(-n // b) for n in lens], wanted + 11, columns)
        return {"op": op, "lens": _ints(lens), "new": _ints(new), "table": table, "free": free,
                "head": _ints([5]), "block": b, "tokens": sum(new) + case["pad"]}
    if op == "append":
        t, h, d, b = case["tokens"], case["heads"], case["dim"], case["block"]
        rows = _normal(g, t, 8 * h * d, scale=1.5)  # the fused projection's rows: q, k and v
        pages = -(-t // b) + 3
        slots = torch.randperm(pages * b, generator=g, device="cuda")[:t].to(torch.int32)
        if case["skip"]:
            slots[torch.rand(t, generator=g, device="cuda") < 0.1] = -1
        caches = []
        for _ in range(2):
            c = _normal(g, pages, b, h, d)
            caches.append(c.to(torch.float8_e4m3fn) if case["e4m3"] else c)
        return {"op": op, "k": rows[:, 6 * h * d:7 * h * d].view(t, h, d),
                "v": rows[:, 7 * h * d:].view(t, h, d), "k_cache": caches[0],
                "v_cache": caches[1], "slots": slots,
                "k_scale": 0.02 if case["e4m3"] else 1.0, "v_scale": 0.03 if case["e4m3"] else 1.0}
    if op == "attn":
        lens, new = _attn_sizes(case)
        h, hk, d, b = case["heads"], case["kv_heads"], case["dim"], case["block"]
        table, _, total = _tables(g, [-(-n // b) for n in lens], 3, -(-max(lens) // b) + 1)
        scale_of = 16.0 if case["e4m3"] else 1.0  # an 8-bit cache is used over more of its range
        caches = []
        for _ in range(2):
            c = _normal(g, total, b, hk, d, scale=scale_of)
            caches.append(c.to(torch.float8_e4m3fn) if case["e4m3"] else c)
        t = sum(new)
        rows = _normal(g, t, (h + 2 * hk) * d, scale=1.5)  # q inside the fused projection's rows
        starts = torch.cumsum(_ints([0] + new), 0).to(torch.int32)
        return {"op": op, "q": rows[:, :h * d].view(t, h, d), "k_cache": caches[0],
                "v_cache": caches[1], "table": table, "starts": starts, "lens": _ints(lens),
                "k_scale": 1 / scale_of, "v_scale": 1 / scale_of, "scale": d ** -0.5,
                "most_new": max(new), "longest": max(lens)}
    m, s, r, n, k = case["rows"], case["adapters"], case["rank"], case["n"], case["k"]
    index, ranks = _lora_index(case)
    return {"op": op, "y": _normal(g, m, n), "x": _normal(g, m, k),
            "a": _normal(g, s, r, k, scale=k ** -0.5), "b": _normal(g, s, n, r, scale=r ** -0.5),
            "index": _ints(index), "ranks": _ints(ranks),
            "scales": torch.rand(s, generator=g, device="cuda") + 0.5}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"plan": _plan, "append": _append, "attn": _attn, "lora": _lora}[state["op"]](state)


def _plan(s):
    if own:
        import nvfp4_weight_only_03_b200 as nv
        p = nv.paged_plan(s["lens"], s["new"], s["table"], s["free"], s["head"], s["block"],
                          tokens=s["tokens"])
        return {"table": s["table"], "starts": p.starts, "lens": p.lens, "slots": p.slots,
                "request": p.request, "positions": p.positions, "head": p.head,
                "missing": p.missing}
    lens, new, table, free, b = s["lens"], s["new"], s["table"], s["free"], s["block"]
    rows, cols = table.shape
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    lens_out = lens + new
    old = (lens + b - 1) // b
    wanted = (lens_out + b - 1) // b
    need = (torch.clamp(wanted, max=cols) - old).clamp(min=0)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(cols, device=lens.device)
    at = s["head"] + first[:, None] + col - old[:, None]
    taken = (col >= old[:, None]) & (col < (old + need)[:, None])
    page = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table.copy_(torch.where(taken, page, table))
    t = torch.arange(s["tokens"], device=lens.device)
    r = torch.searchsorted(ends, t, right=True)
    real = r < rows
    r = r.clamp(max=rows - 1)
    pos = lens[r] + t - starts[r]
    at = pos // b
    page = torch.where(at < cols, table[r, at.clamp(max=cols - 1)], -1)
    slot = torch.where(real & (page >= 0), page * b + pos % b, -1)
    got = torch.minimum(need.sum(), (free.numel() - s["head"]).clamp(min=0))
    i32 = torch.int32
    return {"table": table, "starts": starts.to(i32), "lens": lens_out, "slots": slot.to(i32),
            "request": torch.where(real, r, -1).to(i32),
            "positions": torch.where(real, pos, 0).to(i32),
            "head": (s["head"] + got).to(i32),
            "missing": ((wanted - old).clamp(min=0).sum() - got).to(i32)}


def _append(s):
    if own:
        import nvfp4_weight_only_03_b200 as nv
        nv.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    _put(s["k"], s["k_cache"], s["slots"], s["k_scale"])
    _put(s["v"], s["v_cache"], s["slots"], s["v_scale"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _put(rows, cache, slots, scale):
    keep = slots >= 0
    if cache.dtype == torch.float8_e4m3fn:
        codes = (rows.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        rows, cache = codes.view(torch.uint8), cache.view(torch.uint8)
    cache.view(-1, *cache.shape[2:])[slots[keep].long()] = rows[keep]


def _attn(s):
    if own:
        import nvfp4_weight_only_03_b200 as nv
        return nv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["starts"],
                                  s["lens"], scale=s["scale"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
    q, table, lens, starts = s["q"], s["table"], s["lens"], s["starts"]
    _, b, hk, d = s["k_cache"].shape
    tokens, h, _ = q.shape
    n_new = starts[1:] - starts[:-1]
    i = torch.arange(s["most_new"], device=q.device)
    at = (starts[:-1, None] + i).clamp(max=tokens - 1)
    real = i < n_new[:, None]
    pos = lens[:, None] - n_new[:, None] + i
    j = torch.arange(s["longest"], device=q.device)
    page = table[:, j // b]
    there = (page >= 0) & (j < lens[:, None])
    where = (page.clamp(min=0).long() * b + j % b)
    k = s["k_cache"].view(-1, hk, d)
    v = s["v_cache"].view(-1, hk, d)
    if k.dtype == torch.float8_e4m3fn:
        k, v = k.view(torch.uint8)[where].view(k.dtype), v.view(torch.uint8)[where].view(v.dtype)
    else:
        k, v = k[where], v[where]
    k = k.float()
    v = torch.where(there[:, :, None, None], v.float(), 0.0)
    qg = q[at].float().view(*at.shape, hk, h // hk, d)
    scores = torch.einsum("rihgd,rjhd->rhgij", qg, k) * (s["scale"] * s["k_scale"])
    seen = there[:, None, :] & (j <= pos[:, :, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = scores.sub_(top).exp_()
    total = p.sum(-1)
    o = torch.einsum("rhgij,rjhd->rihgd", p, v) * s["v_scale"]
    o = o / total.permute(0, 3, 1, 2)[..., None].clamp(min=1e-30)
    out = torch.empty(tokens, h, d, dtype=q.dtype, device=q.device)
    out[at[real]] = o.reshape(*at.shape, h, d)[real].to(q.dtype)
    return out


def _lora(s):
    if own:
        import nvfp4_weight_only_03_b200 as nv
        return nv.lora_add(s["y"], s["x"], s["a"], s["b"], s["index"], s["scales"],
                           ranks=s["ranks"])
    a = s["index"].clamp(min=0).long()
    live = torch.arange(s["a"].shape[1], device=a.device) < s["ranks"][a][:, None]
    live &= (s["index"] >= 0)[:, None]
    t = torch.einsum("mrk,mk->mr", s["a"][a].float(), s["x"].float())
    t = torch.where(live, t, 0.0) * s["scales"][a][:, None]
    return (s["y"].float() + torch.einsum("mnr,mr->mn", s["b"][a].float(), t)).to(s["y"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        lens, new = _plan_sizes(case)
        b, n, t = case["block"], len(lens), sum(new)
        taken = sum(-(-(x + y) // b) - -(-x // b) for x, y in zip(lens, new))
        looked = sum(1 for x, y in zip(lens, new) if y and x % b)  # half-filled pages
        # lens and new in; starts and lens out; a page in and out of the list; the tokens' three
        return {"bytes": 4.0 * (2 * n + 2 * n + 1 + 2 * taken + looked + 3 * (t + case["pad"])),
                "flops": 0.0}
    if op == "append":
        values = 2.0 * case["tokens"] * case["heads"] * case["dim"]
        if case["skip"]:
            values *= 0.9
        return {"bytes": values * (3 if case["e4m3"] else 4) + 4 * case["tokens"], "flops": 0.0}
    if op == "attn":
        lens, new = _attn_sizes(case)
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
        cache = 2.0 * sum(lens) * hk * d * (1 if case["e4m3"] else 2)
        tables = 4.0 * sum(-(-n // case["block"]) for n in lens)
        return {"bytes": cache + tables + 4.0 * sum(new) * h * d, "flops": 4.0 * pairs * h * d}
    index, ranks = _lora_index(case)
    n, k = case["n"], case["k"]
    used = sum(ranks[a] for a in set(index) if a >= 0)
    pairs = sum(ranks[a] for a in index if a >= 0)
    return {"bytes": 2.0 * used * (n + k) + 2.0 * case["rows"] * (2 * n + k),
            "flops": 2.0 * pairs * (n + k)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "append":
        outs = {}
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            out = cache.to(torch.float64).view(-1, *cache.shape[2:])
            hit = torch.nonzero(s["slots"] >= 0)[:, 0]
            out[s["slots"][hit].long()] = s[name][hit].double() / s[name + "_scale"]
            outs[name + "_cache"] = out.view(cache.shape)
        return outs
    if op == "lora":
        y, x = s["y"].double(), s["x"].double()
        ranks, scales = s["ranks"].tolist(), s["scales"].tolist()
        for row, a in enumerate(s["index"].tolist()):
            if a >= 0:
                down = s["a"][a, :ranks[a]].double() @ x[row]
                y[row] += scales[a] * (s["b"][a, :, :ranks[a]].double() @ down)
        return y
    _, b, hk, d = s["k_cache"].shape
    group = s["q"].shape[1] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for r, length in enumerate(lens):
        first, count = starts[r], starts[r + 1] - starts[r]
        pages = s["table"][r, :-(-length // b)].long()
        key_at = torch.arange(length, device="cuda")
        for h in range(hk):
            k = s["k_cache"][:, :, h].view(torch.uint8)[pages].view(s["k_cache"].dtype) \
                .reshape(-1, d)[:length].double() * s["k_scale"]
            v = s["v_cache"][:, :, h].view(torch.uint8)[pages].view(s["v_cache"].dtype) \
                .reshape(-1, d)[:length].double() * s["v_scale"]
            for i in range(0, count, 256):
                m = min(256, count - i)
                q = s["q"][first + i:first + i + m, h * group:(h + 1) * group].double()
                w = torch.matmul(q.reshape(-1, d), k.T) * s["scale"]
                row_at = (length - count + i + torch.arange(m, device="cuda"))
                hide = (key_at[None, :] > row_at[:, None]).repeat_interleave(group, 0)
                w = torch.softmax(w.masked_fill_(hide, -math.inf), -1)
                out[first + i:first + i + m, h * group:(h + 1) * group] = \
                    torch.matmul(w, v).view(m, group, d)
    return out
