"""Linear attention with one decay per head, and probabilities from logits, as measured cases.

Operators, each as a user's program calls it:
  fwd     kda_linear_fwd: prompts, of one length or packed one after the other
  step    kda_linear_step: one new token for each sequence, states updated in place
  draft   kda_linear_verify, then kda_linear_commit: drafted tokens, and the states advanced by those that were kept
  bwd     kda_linear_bwd: the gradients of a training step
  logits  kda_logits_probs: penalties, biases, grammar masks and temperature on logits, and their softmax

`own` chooses between the plain forms (elementary torch operations) and the library's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a short prompt, one chunk long: latency
        fwd("fwd short prompt", B=1, T=37, H=32, d=128),
        # the framework's 8k prefill (32 heads of 128), continuing from a state
        fwd("fwd 8k", B=1, T=8192, H=32, d=128, start=True),
        # the framework's packed prefill: four prompts of unequal length, 65536 tokens together
        fwd("fwd packed 64k", B=4, T=65536, H=32, d=128, packed=True),
        # an odd batch with fixed decays, outputs in 32 bits, queries, keys and values side by side in one projection
        fwd("fwd odd batch fp32", B=3, T=2021, H=16, d=64, out="fp32", fixed=True, fused=True, start=True),
        # one request decoding in an idle server: latency
        step("step one request", N=1, H=32, d=128),
        # the framework's decode batch
        step("step 256 requests", N=256, H=32, d=128),
        # verification of 4 drafts (5 tokens a request), then the states advanced by what was kept
        step("drafts of 61 requests", N=61, H=32, d=128, K=5),
        # a training step of the 8k problem
        bwd("bwd 8k", B=1, T=8192, H=32, d=128),
        # a small odd batch, gradients through the initial and the final state
        bwd("bwd odd batch", B=3, T=1001, H=5, d=64, start=True),
        # one request, plain sampling from a small vocabulary: latency
        logits("logits one request", N=1, R=1, V=32768, L=200),
        # the decode batch with 4 drafts each over a large vocabulary, everything switched on
        logits("logits 256 requests", N=256, R=5, V=131072, L=1500, bias=64, mask=True),
        # 16-bit logits and probabilities, an odd vocabulary (rows start at odd addresses), longer drafts
        logits("logits odd 16-bit", N=37, R=8, V=50021, L=4000, bias=7, mask=True, dtype="bf16", out="bf16"),
    ]


def fwd(name, B, T, H, d, out="bf16", packed=False, fixed=False, fused=False, start=False, scale=1.0):
    return dict(name=name, op="fwd", B=B, T=T, H=H, d=d, out=out, packed=packed, fixed=fixed, fused=fused, start=start, scale=scale)


def step(name, N, H, d, K=1, out="fp32", fixed=False):
    return dict(name=name, op="step" if K == 1 else "draft", N=N, K=K, H=H, d=d, out=out, fixed=fixed)


def bwd(name, B, T, H, d, packed=False, start=False, scale=1.0):
    return dict(name=name, op="bwd", B=B, T=T, H=H, d=d, packed=packed, fixed=False, fused=False, start=start, scale=scale)


def logits(name, N, R, V, L, bias=0, mask=False, dtype="fp32", out="fp32", penalties=True):
    return dict(name=name, op="logits", N=N, R=R, V=V, L=L, bias=bias, mask=mask, dtype=dtype, out=out, penalties=penalties)


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "bwd", "logits", "logits"])
    H, d = rng.choice([1, 2, 3, 5, 8, 16, 32, 40, 64]), rng.choice([64, 128, 128])
    if op == "fwd":
        rows = _log(rng, 1, min(200000, 65536 * 32 * 128 // (H * d)))
        B = _log(rng, 1, min(16, rows))
        packed = rng.random() < 0.4
        c = fwd("", B, rows if packed else rows // B, H, d, rng.choice(["bf16", "bf16", "fp32"]), packed, rng.random() < 0.3,
                rng.random() < 0.3, rng.random() < 0.5, rng.choice([1.0, d ** -0.5]))
    elif op == "step":
        N = _log(rng, 1, max(1, min(1024, 256 * 32 * 128 * 128 // (H * d * d))))
        c = step("", N, H, d, rng.choice([1, 1, 2, 5, 8]), rng.choice(["bf16", "fp32", "fp32"]), rng.random() < 0.3)
    elif op == "bwd":
        rows = _log(rng, 1, min(40000, 8192 * 32 * 128 // (H * d)))
        B = _log(rng, 1, min(8, rows))
        packed = rng.random() < 0.3
        c = bwd("", B, rows if packed else rows // B, H, d, packed, rng.random() < 0.5, rng.choice([1.0, d ** -0.5]))
    else:
        V, R = _log(rng, 1000, 200000), rng.randint(1, 8)
        N = max(1, min(_log(rng, 1, 256), 256 * 5 * 131072 // (V * R)))
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        c = logits("", N, R, V, _log(rng, 1, 8000), rng.choice([0, 0, _log(rng, 1, 300)]), rng.random() < 0.4, dtype,
                   rng.choice(["fp32", dtype]), rng.random() < 0.8)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _rows(c):
    return c["T"] if c.get("packed") else c["B"] * c["T"]


def _edges(c, seed):
    """The packed sequences' offsets: cuts drawn from the tokens, on the host."""
    g = torch.Generator().manual_seed(seed)
    T, B = c["T"], c["B"]
    cuts = torch.sort(torch.randperm(T - 1, generator=g)[:B - 1] + 1).values if B > 1 and T > 1 else torch.zeros(B - 1, dtype=torch.long)
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), T)])


def _decays(c, lead, g):
    """Logarithms of the decays: a range of heads from slow to fast, fixed (fp32 [H]) or by token (bf16)."""
    H = c["H"]
    base = torch.exp(torch.linspace(math.log(1e-3), math.log(1.0), H, device="cuda")) if H > 1 else torch.full((1,), 0.02, device="cuda")
    if c["fixed"]:
        return -base * torch.exp(0.1 * torch.randn(H, generator=g, device="cuda"))
    return (-base * torch.exp(torch.randn(lead + (H,), generator=g, device="cuda"))).to(torch.bfloat16)


def _heads(c, lead, g):
    """Queries and keys of unit length, values of unit variance, bf16 [*lead, H, d]."""
    H, d = c["H"], c["d"]
    q, k, v = (torch.randn(lead + (H, d), generator=g, device="cuda") for _ in range(3))
    q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True)) for x in (q, k))
    if c.get("fused"):
        return torch.cat([q, k, v], -2).to(torch.bfloat16).split(H, dim=-2)
    return tuple(x.to(torch.bfloat16) for x in (q, k, v))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = {"case": c}
    if c["op"] == "logits":
        _prepare_logits(c, s, g)
        return s
    if c["op"] in ("fwd", "bwd"):
        N, H, d = c["B"], c["H"], c["d"]
        lead = (c["T"],) if c["packed"] else (c["B"], c["T"])
        s["cu_seqlens"] = _edges(c, seed).to(torch.int32).cuda() if c["packed"] else None
    else:
        N, H, d = c["N"], c["H"], c["d"]
        lead = (N,) if c["op"] == "step" else (N, c["K"])
    s["q"], s["k"], s["v"] = _heads(c, lead, g)
    s["log_alpha"] = _decays(c, lead, g)
    state = 0.02 * torch.randn((N, H, d, d), generator=g, device="cuda")
    if c["op"] in ("step", "draft"):
        s["state"] = state
        if c["op"] == "draft":
            s["accepted"] = torch.randint(0, c["K"] + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
        return s
    s["initial_state"] = state if c["start"] else None
    if c["op"] == "bwd":
        s["d_out"] = torch.randn(lead + (H, d), generator=g, device="cuda").to(torch.bfloat16)
        s["d_final_state"] = torch.randn((N, H, d, d), generator=g, device="cuda") if c["start"] else None
    return s


def _prepare_logits(c, s, g):
    """Logits of a trained model's spread; histories in which some tokens come often."""
    N, R, V, L = c["N"], c["R"], c["V"], c["L"]
    s["logits"] = (3 * torch.randn((N, R, V), generator=g, device="cuda")).to(DT[c["dtype"]])
    s["drafts"] = torch.randint(0, V, (N, R - 1), generator=g, device="cuda", dtype=torch.int32) if R > 1 else None
    s["temperature"] = 0.5 + torch.rand(N, generator=g, device="cuda")
    for name in ("tokens", "lens", "prompt_lens", "repetition", "presence", "frequency", "bias_ids", "bias", "mask"):
        s[name] = None
    if c["penalties"]:
        u = torch.rand((N, L), generator=g, device="cuda")
        s["tokens"] = (V * u ** 4).to(torch.int32).clamp_(max=V - 1)
        s["lens"] = torch.randint(L // 2, L + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
        s["prompt_lens"] = s["lens"] // 2
        s["repetition"] = 1 + 0.3 * torch.rand(N, generator=g, device="cuda")
        s["presence"] = torch.rand(N, generator=g, device="cuda")
        s["frequency"] = 0.1 * torch.rand(N, generator=g, device="cuda")
    if c["bias"]:
        s["bias_ids"] = torch.randint(0, V, (N, c["bias"]), generator=g, device="cuda", dtype=torch.int32)
        s["bias"] = 2 * torch.randn((N, c["bias"]), generator=g, device="cuda")
    if c["mask"]:
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (N, R, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return {"fwd": _own_fwd, "step": _own_step, "draft": _own_draft, "bwd": _own_bwd, "logits": _own_logits}[op](s)
    return {"fwd": _plain_fwd, "step": _plain_step, "draft": _plain_draft, "bwd": _plain_bwd, "logits": _plain_logits}[op](s)


def _own_fwd(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    c = s["case"]
    out, state = kda.kda_linear_fwd(s["q"], s["k"], s["v"], s["log_alpha"], initial_state=s["initial_state"], scale=c["scale"],
                                    out_dtype=DT[c["out"]], cu_seqlens=s["cu_seqlens"])
    return {"out": out, "state": state}


def _own_step(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    out = kda.kda_linear_step(s["q"], s["k"], s["v"], s["log_alpha"], s["state"], out_dtype=DT[s["case"]["out"]])
    return {"out": out, "state": s["state"]}


def _own_draft(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    out = kda.kda_linear_verify(s["q"], s["k"], s["v"], s["log_alpha"], s["state"], out_dtype=DT[s["case"]["out"]])
    kda.kda_linear_commit(s["k"], s["v"], s["log_alpha"], s["state"], s["accepted"])
    return {"out": out, "state": s["state"]}


def _own_bwd(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    g = kda.kda_linear_bwd(s["q"], s["k"], s["v"], s["log_alpha"], s["d_out"], initial_state=s["initial_state"],
                           d_final_state=s["d_final_state"], scale=s["case"]["scale"], cu_seqlens=s["cu_seqlens"])
    if s["initial_state"] is None:
        g.pop("initial_state", None)
    return g


def _own_logits(s):
    import linear_attention_recurrence_fwd_gb300 as kda
    return {"probs": kda.kda_logits_probs(
        s["logits"], tokens=s["tokens"], lens=s["lens"], prompt_lens=s["prompt_lens"], drafts=s["drafts"], repetition=s["repetition"],
        presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"],
        temperature=s["temperature"], out_dtype=DT[s["case"]["out"]])}


def _decayed(q, k, v, log_alpha, start):
    """out_t = sum over s <= t of e^(G_t - G_s) (q_t . k_s) v_s + e^(G_t) start^T q_t, with G the running sum of log_alpha, and the
    state after the last token.  q, k, v [B, T, H, d] fp32, log_alpha [B, T, H]; in chunks, the chunks joined by one product."""
    B, T, H, d = q.shape
    C = min(T, 256 if T <= 16384 else 512)
    n = (T + C - 1) // C
    pad = n * C - T
    # [B, H, n, C, d]; a padded token has no key and no decay
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, n, C, H, d).permute(0, 3, 1, 2, 4) for x in (q, k, v))
    G = torch.nn.functional.pad(log_alpha.double(), (0, 0, 0, pad)).view(B, n, C, H).permute(0, 3, 1, 2).cumsum(-1)
    ends = G[..., -1].cumsum(-1)                                              # [B, H, n]: at each chunk's end
    own_ = torch.matmul((k * torch.exp(G[..., -1:] - G).float()[..., None]).transpose(-1, -2), v)   # [B, H, n, d, d]
    at = torch.arange(n, device="cuda")
    far = (ends - G[..., -1])[..., :, None] - ends[..., None, :]              # from the end of chunk j to the start of chunk i
    far = torch.exp(far.masked_fill(at[None, :] >= at[:, None], -math.inf)).float()
    enter = torch.matmul(far, own_.flatten(-2)).view(B, H, n, d, d)
    if start is not None:
        enter = enter + torch.exp(ends - G[..., -1]).float()[..., None, None] * start[:, :, None]
    last = torch.exp(G[..., -1, -1]).float()[..., None, None] * enter[:, :, -1] + own_[:, :, -1]
    i = torch.arange(C, device="cuda")
    near = (G[..., :, None] - G[..., None, :]).masked_fill(i[None, :] > i[:, None], -math.inf)
    near = torch.exp(near.float()) * torch.matmul(q, k.transpose(-1, -2))
    out = torch.matmul(near, v) + torch.exp(G).float()[..., None] * torch.matmul(q, enter)
    return out.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, d)[:, :T], last


def _padded(s, names):
    """Sequences side by side [B, longest, ...] in fp32, zeros behind each one's end, and where each token lies among them."""
    c = s["case"]
    if not c["packed"]:
        la = s["log_alpha"].float()
        la = la.expand(c["B"], c["T"], c["H"]) if c["fixed"] else la
        return [s[n].float() for n in names], la, None
    cu = s["cu_seqlens"].long()
    lens = cu[1:] - cu[:-1]
    longest = int(lens.max())
    t = torch.arange(longest, device="cuda")
    real = t < lens[:, None]
    index = (cu[:-1, None] + t).clamp(max=c["T"] - 1)
    la = s["log_alpha"].float()
    la = la.expand(c["T"], c["H"]) if c["fixed"] else la
    side = [torch.where(real[..., None, None], s[n].float()[index], 0.0) for n in names]
    return side, torch.where(real[..., None], la[index], 0.0), real


def _plain_fwd(s):
    c = s["case"]
    (q, k, v), la, real = _padded(s, ("q", "k", "v"))
    out, state = _decayed(q * c["scale"], k, v, la, s["initial_state"])
    return {"out": (out if real is None else out[real]).to(DT[c["out"]]), "state": state}


def _plain_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    s["state"].mul_(torch.exp(s["log_alpha"].float())[..., None, None])
    s["state"].add_(k[..., :, None] * v[..., None, :])
    return {"out": (q[..., None, :] @ s["state"])[..., 0, :].to(DT[s["case"]["out"]]), "state": s["state"]}


def _plain_draft(s):
    c = s["case"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    la = s["log_alpha"].float()
    la = la.expand(c["N"], c["K"], c["H"]) if c["fixed"] else la
    out, _ = _decayed(q, k, v, la, s["state"])
    kept = torch.arange(c["K"], device="cuda") < s["accepted"][:, None]
    _, state = _decayed(q, k * kept[..., None, None], v, la * kept[..., None], s["state"])
    s["state"].copy_(state)
    return {"out": out.to(DT[c["out"]]), "state": s["state"]}


def _plain_bwd(s):
    """Each gradient is the operator itself with its arguments in other places, two of them backwards in time."""
    c = s["case"]
    (q, k, v, do), la, real = _padded(s, ("q", "k", "v", "d_out"))
    do = do * c["scale"]
    s0, ds = s["initial_state"], s["d_final_state"]
    dq, last = _decayed(do, v, k, la, None if s0 is None else s0.transpose(-1, -2))
    # backwards, what moves a token's gradient to the one before it is the later token's decay; behind the last one there is none
    back = torch.nn.functional.pad(la[:, 1:], (0, 0, 0, 1)).flip(1)
    do, v, k, q = (x.flip(1) for x in (do, v, k, q))
    dk, first = _decayed(v, do, q, back, None if ds is None else ds.transpose(-1, -2))
    dv, _ = _decayed(k, q, do, back, ds)
    do, v, k, q, dk, dv = (x.flip(1) for x in (do, v, k, q, dk, dv))
    last = last.transpose(-1, -2)
    part = (q * dq).sum(-1).double() - (k * dk).sum(-1).double()
    dla = part.flip(1).cumsum(1).flip(1)
    if ds is not None:
        dla = dla + (last.double() * ds.double()).sum((-1, -2))[:, None]
    out = {"q": dq, "k": dk, "v": dv, "log_alpha": dla}
    out = {n: (x if real is None else x[real]).to(torch.bfloat16) for n, x in out.items()}
    if s0 is not None:
        out["initial_state"] = torch.exp(la[:, 0])[..., None, None] * first.transpose(-1, -2)
    return out


def _counts(s, V):
    """How often each token was said before each row, in the whole history [N, R, V] and without the prompt."""
    c = s["case"]
    N, R = c["N"], c["R"]
    at = torch.arange(c["L"], device="cuda")
    tok = s["tokens"].long()
    whole, new = (torch.zeros((N, V), device="cuda") for _ in range(2))
    held = at < s["lens"][:, None]
    whole.scatter_add_(1, tok, held.float())
    new.scatter_add_(1, tok, (held & (at >= s["prompt_lens"][:, None])).float())
    whole, new = (x[:, None].repeat(1, R, 1) for x in (whole, new))
    if R > 1:
        # draft i has been said before the rows i + 1 and later
        said = torch.zeros((N, R, V), device="cuda")
        said[:, 1:].scatter_add_(2, s["drafts"].long()[..., None], torch.ones((N, R - 1, 1), device="cuda"))
        said = said.cumsum(1)
        whole, new = whole + said, new + said
    return whole, new


def _plain_logits(s):
    c = s["case"]
    x = s["logits"].float()
    V = c["V"]
    if c["penalties"]:
        whole, new = _counts(s, V)
        rep, pres, freq = (s[n][:, None, None] for n in ("repetition", "presence", "frequency"))
        x = torch.where(whole > 0, torch.where(x > 0, x / rep, x * rep), x)
        del whole
        x = x - freq * new - torch.where(new > 0, pres, 0.0)
        del new
    if c["bias"]:
        extra = torch.zeros((c["N"], V), device="cuda").scatter_add_(1, s["bias_ids"].long(), s["bias"])
        x = x + extra[:, None]
    if c["mask"]:
        bit = torch.arange(V, device="cuda")
        allowed = ((s["mask"][..., bit // 32] >> (bit % 32).int()) & 1) != 0
        x = x.masked_fill(~allowed, -math.inf)
    x = x / s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    return {"probs": (x / torch.where(total > 0, total, 1.0)).to(DT[c["out"]])}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "logits":
        rows = c["N"] * c["R"]
        held = rows * c["V"] * (SIZE[c["dtype"]] + SIZE[c["out"]] + (0.125 if c["mask"] else 0))
        return {"bytes": held + c["N"] * (4 * c["L"] * c["penalties"] + 8 * c["bias"]), "flops": 8.0 * rows * c["V"]}
    H, d = c["H"], c["d"]
    decay = 0 if c["fixed"] else 2
    if c["op"] in ("step", "draft"):
        n = c["N"] * H
        return {"bytes": n * (8 * d * d + c["K"] * (d * (6 + SIZE[c["out"]]) + decay)), "flops": 5.0 * n * c["K"] * d * d}
    rows, states = _rows(c) * H, c["B"] * H * 4 * d * d
    if c["op"] == "fwd":
        # two products of a token with the state, and half of two products with 64 tokens around it
        return {"bytes": rows * (6 * d + SIZE[c["out"]] * d + decay) + states * (1 + c["start"]), "flops": rows * (4.0 * d * d + 128.0 * d)}
    return {"bytes": rows * (14 * d + 2 * decay) + states * 3 * c["start"], "flops": rows * (10.0 * d * d + 320.0 * d)}


# ---------------------------------------------------------------- the definitions in 64 bits, token by token

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "logits":
        return _exact_logits(s, c) if c["N"] * c["R"] * c["V"] <= 1 << 28 else None
    if c["op"] in ("step", "draft"):
        return _exact_step(s, c)
    if c["T"] > (140000 if c["op"] == "fwd" else 40000):
        return None
    return (_exact_fwd if c["op"] == "fwd" else _exact_bwd)(s, c)


def _sequences(s, c):
    """Each sequence's rows: slices of the tokens, all at once where they have one length."""
    if not c["packed"]:
        return [(slice(None), slice(None))]
    cu = s["cu_seqlens"].tolist()
    return [(slice(a, b), slice(n, n + 1)) for n, (a, b) in enumerate(zip(cu[:-1], cu[1:]))]


def _tokens_first(s, c, where):
    """The tensors of _sequences' rows as [T, B, H, ...] in 64 bits."""
    got = []
    for n in ("q", "k", "v", "log_alpha") + (("d_out",) if "d_out" in s else ()):
        x = s[n].double()
        if n == "log_alpha" and c["fixed"]:
            x = x.expand(s["q"].shape[:-1])
        got.append(x[where][:, None] if c["packed"] else x.transpose(0, 1))
    return got


def _exact_fwd(s, c):
    B, H, d = c["B"], c["H"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    state = torch.zeros((B, H, d, d), dtype=torch.float64, device="cuda")
    if s["initial_state"] is not None:
        state += s["initial_state"].double()
    for where, n in _sequences(s, c):
        q, k, v, la = _tokens_first(s, c, where)
        a, S = torch.exp(la), state[n].clone()
        for t in range(q.shape[0]):
            S.mul_(a[t][..., None, None]).addcmul_(k[t][..., :, None], v[t][..., None, :])
            o = torch.matmul(q[t][..., None, :], S)[..., 0, :]
            if c["packed"]:
                out[where.start + t] = o[0]
            else:
                out[:, t] = o
        state[n] = S
    return {"out": out * c["scale"], "state": state}


def _exact_step(s, c):
    q, k, v, la = (s[n].double() for n in ("q", "k", "v", "log_alpha"))
    S = s["state"].double()
    if c["op"] == "step":
        S = torch.exp(la)[..., None, None] * S + torch.einsum("nhk,nhv->nhkv", k, v)
        return {"out": torch.einsum("nhk,nhkv->nhv", q, S), "state": S}
    la = la.expand(q.shape[:-1])
    kept, outs = S.clone(), []
    for t in range(c["K"]):
        S = torch.exp(la[:, t])[..., None, None] * S + torch.einsum("nhk,nhv->nhkv", k[:, t], v[:, t])
        outs.append(torch.einsum("nhk,nhkv->nhv", q[:, t], S))
        kept = torch.where((s["accepted"] > t)[:, None, None, None], S, kept)
    return {"out": torch.stack(outs, 1), "state": kept}


def _exact_bwd(s, c):
    """The recurrence backwards; a decay's gradient as <the state it acts on, the gradient that arrives there>, every 64 states held."""
    B, H, d = c["B"], c["H"], c["d"]
    grads = {n: torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")}
    grads["log_alpha"] = torch.zeros(s["q"].shape[:-1], dtype=torch.float64, device="cuda")
    d0 = torch.zeros((B, H, d, d), dtype=torch.float64, device="cuda")
    for where, n in _sequences(s, c):
        q, k, v, la, do = _tokens_first(s, c, where)
        do, a, T = do * c["scale"], torch.exp(la), q.shape[0]
        S = torch.zeros_like(d0[n]) if s["initial_state"] is None else s["initial_state"][n].double()
        held = []
        for t in range(T):
            if t % 64 == 0:
                held.append(S)
            S = torch.addcmul(a[t][..., None, None] * S, k[t][..., :, None], v[t][..., None, :])
        G = torch.zeros_like(d0[n]) if s["d_final_state"] is None else s["d_final_state"][n].double().clone()
        part = {m: [None] * T for m in grads}
        for block in range((T - 1) // 64, -1, -1):
            S, before = held[block], []
            for t in range(64 * block, min(T, 64 * block + 64)):
                before.append(S)
                S = torch.addcmul(a[t][..., None, None] * S, k[t][..., :, None], v[t][..., None, :])
            for t in range(min(T, 64 * block + 64) - 1, 64 * block - 1, -1):
                part["q"][t] = torch.matmul(S, do[t][..., None])[..., 0]
                G.addcmul_(q[t][..., :, None], do[t][..., None, :])
                part["k"][t] = torch.matmul(G, v[t][..., None])[..., 0]
                part["v"][t] = torch.matmul(k[t][..., None, :], G)[..., 0, :]
                S = before[t - 64 * block]
                G.mul_(a[t][..., None, None])
                part["log_alpha"][t] = (S * G).sum((-1, -2))
        for m in grads:
            x = torch.stack(part[m])
            if c["packed"]:
                grads[m][where] = x[:, 0]
            else:
                grads[m].copy_(x.transpose(0, 1))
        d0[n] = G
    if s["initial_state"] is not None:
        grads["initial_state"] = d0
    return grads


def _exact_logits(s, c):
    """Row by row."""
    N, R, V = c["N"], c["R"], c["V"]
    out = torch.zeros((N, R, V), dtype=torch.float64, device="cuda")
    ids = torch.arange(V, device="cuda")
    for n in range(N):
        if c["penalties"]:
            L, P = int(s["lens"][n]), int(s["prompt_lens"][n])
            rep, pres, freq = (float(s[m][n]) for m in ("repetition", "presence", "frequency"))
            prompt = torch.bincount(s["tokens"][n, :min(L, P)].long(), minlength=V)
            new = torch.bincount(s["tokens"][n, P:L].long(), minlength=V)
        if c["bias"]:
            extra = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, s["bias_ids"][n].long(), s["bias"][n].double())
        for r in range(R):
            x = s["logits"][n, r].double()
            if c["penalties"]:
                if r:
                    new[s["drafts"][n, r - 1].long()] += 1
                x = torch.where(prompt + new > 0, torch.where(x > 0, x / rep, x * rep), x) - freq * new - pres * (new > 0)
            if c["bias"]:
                x = x + extra
            if c["mask"]:
                word = s["mask"][n, r].long() & 0xffffffff
                x = torch.where((word[ids // 32] >> (ids % 32)) & 1 == 1, x, -math.inf)
            x = x / float(s["temperature"][n])
            if bool((x > -math.inf).any()):
                out[n, r] = torch.softmax(x, -1)
    return {"probs": out}
