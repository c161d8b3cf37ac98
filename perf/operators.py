"""The serving operators that surround the recurrent layer in a hybrid stack, as measured cases.

Three operators, each as a user's program calls it:
  append  kda_cache_append: new keys and values into a paged cache, rotated by position on the way (queries too)
  attend  kda_cache_attend: the newest tokens of each sequence over that cache
  accept  kda_draft_accept: drafted tokens checked against the target's probabilities

`own` chooses between the plain forms (elementary torch operations) and the library's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # one request in an idle server, a short chat: latency only
        attend("attend one short request", N=1, lo=200, hi=200, Hq=32, Hkv=8, d=128, page=16),
        # the framework's decode batch (256 sequences, 32 heads of 128), lengths as mixed traffic has them
        attend("attend 256 ragged requests", N=256, lo=7, hi=8191, Hq=32, Hkv=8, d=128, page=64),
        # one request with a million tokens and few key heads: all the parallelism is along the length
        attend("attend one request of 1M", N=1, lo=1048575, hi=1048575, Hq=16, Hkv=2, d=128, page=64),
        # verification of 4 drafts (5 tokens a request) over an 8-bit cache, 40 query rows to a key head
        attend("attend 5 tokens 8-bit cache", N=32, K=5, lo=1000, hi=32000, Hq=32, Hkv=4, d=128, page=32, cache="e4m3"),
        # heads of 64 without sharing, a window of odd length, pages of 48 tokens laid out head by head
        attend("attend window heads of 64", N=45, K=2, lo=0, hi=5003, Hq=16, Hkv=16, d=64, page=48, act="fp16", cache="fp16",
               window=1001, layout="head", short=True),
        # one decode step of the 256-sequence batch
        append("append one token each", N=256, K=1, far=8191, Hq=32, Hkv=8, d=128, page=64, rot=128),
        # the drafts of a verification at far positions, half the channels rotated in neighbouring pairs, 8-bit cache
        append("append drafts 8-bit far", N=61, K=5, far=1048000, Hq=32, Hkv=4, d=128, page=32, rot=64, pairs=True, cache="e4m3", short=True),
        # packed prompts of 65536 tokens in 4 sequences (the framework's packed prefill)
        append("append packed prompts", N=4, K=0, T=65536, far=0, Hq=32, Hkv=8, d=128, page=64, rot=128),
        # a short prompt chunk after a cached prefix, heads of 64, head-by-head pages, no rotation
        append("append chunk no rotation", N=3, K=0, T=1021, far=3000, Hq=16, Hkv=16, d=64, page=48, rot=0, act="fp16", cache="fp16", layout="head"),
        # one request, one vocabulary row: latency
        accept("accept one request", N=1, K=4, V=32768),
        # the 256-sequence batch over a large vocabulary
        accept("accept 256 requests", N=256, K=4, V=131072),
        # 16-bit probabilities, odd vocabulary (rows start at odd addresses), longer drafts of unequal length
        accept("accept odd 16-bit", N=37, K=7, V=50021, prob="bf16", short=True),
    ]


def attend(name, N, lo, hi, Hq, Hkv, d, page, K=1, act="bf16", cache="bf16", window=0, layout="token", short=False):
    return dict(name=name, op="attend", N=N, K=K, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, act=act, cache=cache,
                window=window, layout=layout, short=short)


def append(name, N, K, far, Hq, Hkv, d, page, rot, T=0, pairs=False, act="bf16", cache="bf16", layout="token", short=False):
    return dict(name=name, op="append", N=N, K=K, T=T, far=far, Hq=Hq, Hkv=Hkv, d=d, page=page, rot=rot, pairs=pairs, act=act,
                cache=cache, layout=layout, short=short)


def accept(name, N, K, V, prob="fp32", short=False, point=False):
    return dict(name=name, op="accept", N=N, K=K, V=V, prob=prob, short=short, point=point)


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "accept"])
    if op == "accept":
        V = _log(rng, 1000, 200000)
        N, K = _log(rng, 1, 256), rng.randint(1, 8)
        N = max(1, min(N, 256 * 9 * 131072 // (V * (2 * K + 1)) ))
        c = accept("", N, K, V, rng.choice(["fp32", "fp32", "bf16"]), rng.random() < 0.3, rng.random() < 0.2)
    else:
        act = rng.choice(["bf16", "bf16", "fp16"])
        cache = rng.choice([act, act, "e4m3"])
        d, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16] if Hkv <= 4 else [1, 2, 4])
        page, layout = rng.choice([8, 16, 32, 48, 64, 100, 128]), rng.choice(["token", "token", "head"])
        if op == "attend":
            N = _log(rng, 1, 256)
            most = min(1 << 20, (256 * 8192 * 8 * 128) // (N * Hkv * d))
            hi = _log(rng, 1, most)
            lo = rng.choice([hi, rng.randint(0, hi), 0])
            K = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
            c = attend("", N, lo, hi, Hq, Hkv, d, page, K, act, cache, rng.choice([0, 0, 0, _log(rng, 1, 5000)]), layout,
                       rng.random() < 0.2)
        else:
            rot = rng.choice([0, d // 2, d, d])
            far = rng.choice([0, _log(rng, 1, 1 << 20)])
            if rng.random() < 0.5:
                c = append("", _log(rng, 1, 512), rng.randint(1, 8), far, Hq, Hkv, d, page, rot, 0, rng.random() < 0.4, act,
                           cache, layout, rng.random() < 0.2)
            else:
                T = _log(rng, 1, 65536 * 40 * 128 // (max(40, Hq + Hkv) * 128))
                c = append("", min(T, _log(rng, 1, 64)), 0, far, Hq, Hkv, d, page, rot, T, rng.random() < 0.4, act, cache, layout)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _lens(c):
    """The sequences' lengths before the new tokens: evenly spaced, so that a case's work is the same for every seed."""
    N, lo, hi = c["N"], c["lo"], c["hi"]
    return [lo + (hi - lo) * n // max(1, N - 1) for n in range(N)]


def _pool(c, pages, g):
    shape = (pages, c["Hkv"], c["page"], c["d"]) if c["layout"] == "head" else (pages, c["page"], c["Hkv"], c["d"])
    x = torch.empty(shape, dtype=DT[c["cache"]], device="cuda")
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 28):  # in pieces: the fp32 numbers of a whole pool need not fit
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return x.transpose(1, 2) if c["layout"] == "head" else x


def _counts(c, g):
    if not c["short"]:
        return None
    return torch.randint(0, c["K"] + 1, (c["N"],), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s = {"case": c}
    if c["op"] == "accept":
        _prepare_accept(c, s, g)
        return s
    if c["op"] == "attend":
        host = torch.tensor(_lens(c))[torch.randperm(c["N"], generator=torch.Generator().manual_seed(seed))]
        first, new = torch.zeros_like(host), torch.full_like(host, c["K"])
        s["q"] = (1.5 * torch.randn((c["N"], c["K"], c["Hq"], c["d"]), generator=g, device="cuda")).to(DT[c["act"]])
        s["counts"] = _counts(c, g)
        s["window"] = c["window"]
    else:
        rng = torch.Generator().manual_seed(seed)
        host = torch.randint(0, c["far"] + 1, (c["N"],), generator=rng)
        if c["K"]:
            T, new = c["N"] * c["K"], torch.full_like(host, c["K"])
            s["cu_seqlens"], s["counts"] = None, _counts(c, g)
        else:
            T = c["T"]
            cuts = torch.sort(torch.randperm(T - 1, generator=rng)[:c["N"] - 1] + 1).values if c["N"] > 1 else torch.zeros(0, dtype=torch.long)
            edges = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), T)])
            new = edges[1:] - edges[:-1]
            s["cu_seqlens"], s["counts"] = edges.to(torch.int32).cuda(), None
        first = host // c["page"]
        # the projection's output, queries, keys and values of a token side by side
        fused = torch.randn((T, (c["Hq"] + 2 * c["Hkv"]) * c["d"]), generator=g, device="cuda").to(DT[c["act"]])
        lead = (c["N"], c["K"]) if c["K"] else (T,)
        q, k, v = fused.split([c["Hq"] * c["d"], c["Hkv"] * c["d"], c["Hkv"] * c["d"]], dim=1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, c["d"])).unflatten(0, lead) if c["K"] else x.unflatten(1, (-1, c["d"]))
                                  for x in (q, k, v))
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).cuda() if c["rot"] else None
    # pages from `first` to the last new token, handed out in random order; -1 where a request holds none
    last = (host + new - 1) // c["page"]
    need = (last - first + 1).clamp(min=0)
    # as many for every seed: a request's tokens touch one page more where they start late in a page
    total = int(need.sum()) if c["op"] == "attend" else c["N"] * ((c["K"] - 2) // c["page"] + 2) if c["K"] else c["T"] // c["page"] + 2 * c["N"]
    at = torch.arange(int(last.max()) + 1).expand(c["N"], -1)
    held = (at >= first[:, None]) & (at <= last[:, None])
    table = torch.full(at.shape, -1, dtype=torch.int32, device="cuda")
    table[held.cuda()] = torch.randperm(total, generator=g, device="cuda")[:int(need.sum())].to(torch.int32)
    s["k_pages"], s["v_pages"] = _pool(c, total, g), _pool(c, total, g)
    s["table"], s["lens"] = table, host.to(torch.int32).cuda()
    s["k_scale"], s["v_scale"] = (0.5, 0.25) if c["cache"] == "e4m3" else (1.0, 1.0)
    if own:
        import linear_attention_recurrence_fwd_gb300 as kda
        s["cache"] = kda.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lens"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


def _prepare_accept(c, s, g):
    """Probabilities as a softmax gives them, the draft model's near the target's, drafts drawn from the draft model."""
    N, K, V = c["N"], c["K"], c["V"]
    p = torch.empty((N, K + 1, V), dtype=DT[c["prob"]], device="cuda")
    q = torch.empty((N, K, V), dtype=DT[c["prob"]], device="cuda")
    toks = torch.empty((N, K), dtype=torch.int32, device="cuda")
    step = max(1, (1 << 28) // ((K + 1) * V))
    for n in range(0, N, step):
        z = 3 * torch.randn((min(step, N - n), K + 1, V), generator=g, device="cuda")
        p[n:n + step] = torch.softmax(z, -1)
        z = z[:, :K] + 0.5 * torch.randn(z[:, :K].shape, generator=g, device="cuda")
        z = torch.softmax(z, -1)
        q[n:n + step] = z
        race = z / torch.empty_like(z).exponential_(generator=g)
        toks[n:n + step] = race.argmax(-1).to(torch.int32)
    s["target"], s["draft"], s["tokens"] = p, None if c["point"] else q, toks
    s["uniform"] = torch.rand((N, K + 1), generator=g, device="cuda")
    s["draft_lens"] = torch.randint(-1, K + 1, (N,), generator=g, device="cuda", dtype=torch.int32) if c["short"] else None


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "accept": _own_accept}[op](s)
    return {"attend": _plain_attend, "append": _plain_append, "accept": _plain_accept}[op](s)


def _own_attend(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    out, lse = kda.kda_cache_attend(s["q"], s["cache"], window=s["window"], counts=s["counts"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_append(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    q = kda.kda_cache_append(s["k"], s["v"], s["cache"], q=s["q"], inv_freq=s["inv_freq"], interleaved=s["case"]["pairs"],
                             cu_seqlens=s["cu_seqlens"], counts=s["counts"])
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_accept(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    counts, tokens = kda.kda_draft_accept(s["tokens"], s["draft"], s["target"], s["uniform"], draft_lens=s["draft_lens"])
    return {"counts": counts, "tokens": tokens}


def _plain_attend(s):
    q, lens = s["q"], s["lens"].long()
    N, K, Hq, d = q.shape
    Hkv = s["k_pages"].shape[2]
    at = s["table"].long().clamp(min=0)
    L = at.shape[1] * s["k_pages"].shape[1]
    last = lens[:, None] + torch.arange(K, device="cuda")                       # each query's own position
    real = torch.ones_like(last, dtype=torch.bool) if s["counts"] is None else torch.arange(K, device="cuda") < s["counts"][:, None]
    pos = torch.arange(L, device="cuda")
    seen = (pos <= last[..., None]) & real[..., None]                           # [N, K, L]
    if s["window"]:
        seen = seen & (pos > last[..., None] - s["window"])
    used = seen.any(1)[..., None, None]
    k = s["k_pages"][at].reshape(N, L, Hkv, d).float().masked_fill(~used, 0)
    x = torch.matmul(_rows(q, Hkv).float(), k.permute(0, 2, 3, 1))              # [N, Hkv, K G, L]
    del k
    x = x.view(N, Hkv, K, Hq // Hkv, L) * (s["k_scale"] / math.sqrt(d))
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    v = s["v_pages"][at].reshape(N, L, Hkv, d).float().masked_fill(~used, 0)
    o = torch.matmul(x.view(N, Hkv, -1, L), v.permute(0, 2, 1, 3)).view(N, Hkv, K, Hq // Hkv, d)
    o = torch.where(total > 0, o * s["v_scale"] / total, 0.0)
    lse = torch.log(total) + top
    return {"out": o.transpose(1, 2).reshape(N, K, Hq, d).to(q.dtype), "lse": lse[..., 0].transpose(1, 2).reshape(N, K, Hq)}


def _rows(q, Hkv):
    """[N, K, Hq, d] to [N, Hkv, K G, d]: the query rows of each key head."""
    N, K, Hq, d = q.shape
    return q.view(N, K, Hkv, Hq // Hkv, d).transpose(1, 2).reshape(N, Hkv, -1, d)


def _owner(s, T):
    """Each token's sequence and its number in it."""
    t = torch.arange(T, device="cuda")
    if s["cu_seqlens"] is None:
        K = s["case"]["K"]
        return t // K, t % K
    n = torch.searchsorted(s["cu_seqlens"][1:].long(), t, right=True)
    return n, t - s["cu_seqlens"].long()[n]


def _rotate(x, pos, inv_freq, pairs):
    """[T, H, d] in fp32, rotated by the angles pos * inv_freq (64 bits: a far position's angle has many turns)."""
    if inv_freq is None:
        return x
    a = pos.double()[:, None] * inv_freq
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    R = 2 * inv_freq.numel()
    u, w = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    y, z = u * cos - w * sin, u * sin + w * cos
    y = torch.stack([y, z], -1).flatten(-2) if pairs else torch.cat([y, z], -1)
    return torch.cat([y, x[..., R:]], -1)


def _store(x, scale, dtype):
    x = x / scale
    return x.clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _plain_append(s):
    c = s["case"]
    q, k, v = (s[n].reshape(-1, s[n].shape[-2], c["d"]).float() for n in ("q", "k", "v"))
    n, i = _owner(s, q.shape[0])
    pos = s["lens"].long()[n] + i
    q, k = (_rotate(x, pos, s["inv_freq"], c["pairs"]) for x in (q, k))
    page, row = s["table"].long()[n, pos // c["page"]], pos % c["page"]
    if s["counts"] is not None:
        real = i < s["counts"][n]
        page, row, k, v = page[real], row[real], k[real], v[real]
    s["k_pages"][page, row] = _store(k, s["k_scale"], s["k_pages"].dtype)
    s["v_pages"][page, row] = _store(v, s["v_scale"], s["v_pages"].dtype)
    return {"q": q.to(s["q"].dtype).view(s["q"].shape), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_accept(s):
    p, u, tok = s["target"], s["uniform"].double(), s["tokens"].long()
    N, K = tok.shape
    V = p.shape[-1]
    lens = torch.full((N,), K, device="cuda") if s["draft_lens"] is None else s["draft_lens"].long()
    pt = p[:, :K].gather(2, tok[..., None])[..., 0].double()
    qt = torch.ones_like(pt) if s["draft"] is None else s["draft"].gather(2, tok[..., None])[..., 0].double()
    ok = (u[:, :K] * qt < pt) & (torch.arange(K, device="cuda") < lens[:, None])
    a = ok.long().cumprod(1).sum(1)                                             # drafts taken
    rows = torch.arange(N, device="cuda")
    top = p[rows, a].double()
    if s["draft"] is None:
        low = torch.zeros_like(top).scatter_(1, tok[rows, a.clamp(max=K - 1), None], math.inf)
    else:
        low = s["draft"][rows, a.clamp(max=K - 1)].double()
    w = torch.where((a < lens)[:, None], (top - low).clamp(min=0), top)
    w = torch.where((w.sum(1) > 0)[:, None], w, top)
    run_ = w.cumsum(1)
    nxt = (run_ <= u[:, K:] * run_[:, -1:]).sum(1).clamp(max=V - 1)
    i = torch.arange(K + 1, device="cuda")
    out = torch.where(i < a[:, None], torch.nn.functional.pad(tok, (0, 1)), torch.where(i == a[:, None], nxt[:, None], -1))
    idle = lens < 0
    return {"counts": torch.where(idle, 0, a + 1).int(), "tokens": torch.where(idle[:, None], -1, out).int()}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "accept":
        # the last row of probabilities, and for about two requests in three a row of the draft model's
        rows = 1.0 if c["point"] else 1.65
        return {"bytes": c["N"] * (rows * c["V"] * SIZE[c["prob"]] + 12 * c["K"]), "flops": c["N"] * 3.0 * c["V"]}
    if c["op"] == "append":
        T = c["N"] * c["K"] or c["T"]
        row = c["d"] * SIZE[c["act"]]
        moved = T * (2 * c["Hq"] * row + 2 * c["Hkv"] * (row + c["d"] * SIZE[c["cache"]]))
        return {"bytes": moved, "flops": 3.0 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    share = 0.5 if c["short"] else 1.0
    seen = [min(n + c["K"], c["window"] + c["K"] - 1) if c["window"] else n + c["K"] for n in _lens(c)]
    tokens = float(sum(seen))
    io = 2 * c["N"] * c["K"] * c["Hq"] * c["d"] * SIZE[c["act"]]
    return {"bytes": 2 * tokens * c["Hkv"] * c["d"] * SIZE[c["cache"]] + io, "flops": 4 * share * tokens * c["K"] * c["Hq"] * c["d"]}


# ---------------------------------------------------------------- the definitions in 64 bits, sequence by sequence

def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "accept": _exact_accept}[case["op"]](s, case)


def _exact_attend(s, c):
    N, K, Hq, d = s["q"].shape
    G = Hq // c["Hkv"]
    out = torch.zeros((N, K, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((N, K, Hq), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    counts = [K] * N if s["counts"] is None else s["counts"].tolist()
    for n in range(N):
        held = s["table"][n, :(lens[n] + K - 1) // c["page"] + 1].long()
        keys, values = (x[held].flatten(0, 1) for x in (s["k_pages"], s["v_pages"]))
        for i in range(counts[n]):
            end = lens[n] + i + 1
            start = max(0, end - c["window"]) if c["window"] else 0
            k, v = keys[start:end].double() * s["k_scale"], values[start:end].double() * s["v_scale"]
            q = s["q"][n, i].double().view(c["Hkv"], G, d)
            x = torch.bmm(q, k.permute(1, 2, 0)) / math.sqrt(d)
            out[n, i] = torch.bmm(torch.softmax(x, -1), v.transpose(0, 1)).view(Hq, d)
            lse[n, i] = torch.logsumexp(x, -1).view(Hq)
    return {"out": out, "lse": lse}


def _exact_append(s, c):
    """Rotation as a product of complex numbers; the pages' values before the rounding to their type."""
    lens = s["lens"].tolist()
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    counts = None if s["counts"] is None else s["counts"].tolist()
    edges = [n * c["K"] for n in range(c["N"] + 1)] if c["K"] else s["cu_seqlens"].tolist()
    q, k, v = (s[n].reshape(-1, s[n].shape[-2], c["d"]).double() for n in ("q", "k", "v"))
    half = c["rot"] // 2
    for n in range(c["N"]):
        a, b = edges[n], edges[n + 1]
        pos = lens[n] + torch.arange(b - a, device="cuda")
        if half:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None].double() * s["inv_freq"])[:, None]
            for x in (q, k):
                part = x[a:b, :, :c["rot"]]
                if c["pairs"]:
                    z = torch.view_as_complex(part.unflatten(-1, (half, 2)).contiguous()) * turn
                    x[a:b, :, :c["rot"]] = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
                    x[a:b, :, :half], x[a:b, :, half:c["rot"]] = z.real, z.imag
        m = (b - a) if counts is None else counts[n]
        page, row = s["table"][n].long()[pos[:m] // c["page"]], pos[:m] % c["page"]
        kp[page, row], vp[page, row] = k[a:a + m] / s["k_scale"], v[a:a + m] / s["v_scale"]
    return {"q": q.view(s["q"].shape), "k_pages": kp, "v_pages": vp}


def _exact_accept(s, c):
    """Each request by itself; whole numbers, held to be equal."""
    N, K, V = c["N"], c["K"], c["V"]
    u, tok = s["uniform"].double().tolist(), s["tokens"].tolist()
    lens = [K] * N if s["draft_lens"] is None else s["draft_lens"].tolist()
    counts, tokens = [], []
    for n in range(N):
        if lens[n] < 0:
            counts.append(0)
            tokens.append([-1] * (K + 1))
            continue
        a = 0
        while a < lens[n]:
            t = tok[n][a]
            q = 1.0 if s["draft"] is None else float(s["draft"][n, a, t])
            if not u[n][a] * q < float(s["target"][n, a, t]):
                break
            a += 1
        w = s["target"][n, a].double()
        if a < lens[n]:
            if s["draft"] is None:
                rest = w.clone()
                rest[tok[n][a]] = 0
            else:
                rest = torch.relu(w - s["draft"][n, a].double())
            w = rest if float(rest.sum()) > 0 else w
        total = torch.cumsum(w, 0)
        at = int(torch.searchsorted(total, u[n][K] * total[-1], right=True))
        counts.append(a + 1)
        tokens.append(tok[n][:a] + [min(at, V - 1)] + [-1] * (K - a))
    return {"counts": torch.tensor(counts, dtype=torch.int32), "tokens": torch.tensor(tokens, dtype=torch.int32)}
