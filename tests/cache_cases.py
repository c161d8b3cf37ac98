"""Inputs and 64-bit references shared by the tests of the calls around a
paged cache.  Tolerances count roundings: half a step of the output's type,
`torch.finfo(t).eps / 2` relative, and the fp32 sums of the kernels."""
import math

import torch

from linear_attention_recurrence_fwd_gb300 import binding

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32,
                                            torch.float8_e4m3fn)}
NAN = float("nan")


def make_cache(lens, K, Hkv, d, page, dtype, seed=0, layout="token", width=None, k_scale=1.0,
               v_scale=1.0, spare=3, fill=NAN):
    """A cache whose sequences hold lens[n] + K tokens on pages in random
    order; whatever no sequence holds is `fill`, table entries of no page are
    -1.  Returns (cache, keys, values): the lists of each sequence's tokens,
    on the host in fp64 as stored values times scale."""
    g = torch.Generator().manual_seed(seed)
    need = [max(0, (n + K + page - 1) // page) for n in lens]
    total = sum(need) + spare
    width = max([1] + need) if width is None else width
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    shape = (total, Hkv, page, d) if layout == "head" else (total, page, Hkv, d)
    pools = []
    for _ in range(2):
        x = torch.full(shape, fill, dtype=torch.float32)
        pools.append(x.transpose(1, 2) if layout == "head" else x)
    keys, values, at = [], [], 0
    for n, (length, pages) in enumerate(zip(lens, need)):
        held = order[at:at + pages]
        at += pages
        table[n, :pages] = held.to(torch.int32)
        rows = []
        for x, scale in zip(pools, (k_scale, v_scale)):
            tok = torch.randn((max(0, length + K), Hkv, d), generator=g).to(dtype).float()
            pos = torch.arange(tok.shape[0])
            if tok.shape[0]:
                x[held[pos // page], pos % page] = tok
            rows.append(tok.double() * scale)
        keys.append(rows[0])
        values.append(rows[1])
    kp, vp = (x.to(dtype).cuda() if layout == "token" else
              x.transpose(1, 2).to(dtype).cuda().transpose(1, 2) for x in pools)
    cache = binding.PagedCache(kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                               k_scale=k_scale, v_scale=v_scale)
    return cache, keys, values


def attend_reference(q, keys, values, lens, counts, scale, window):
    """fp64 on the host.  Returns (out, lse, tolerance of out, of lse); the
    tolerances hold for fp32 scores, 16-bit weights and one rounding at the end."""
    N, K, Hq, d = q.shape
    half = HALF[q.dtype]
    q = q.double().cpu()
    out = torch.zeros((N, K, Hq, d), dtype=torch.float64)
    lse = torch.full((N, K, Hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for n in range(N):
        k, v = keys[n], values[n]
        for i in range(K if counts is None else counts[n]):
            end = lens[n] + i + 1
            start = max(0, end - window) if window else 0
            if end <= start:
                continue
            Hkv = k.shape[1]
            qq = q[n, i].view(Hkv, Hq // Hkv, d)
            kk, vv = k[start:end].permute(1, 2, 0), v[start:end].transpose(0, 1)
            x = qq @ kk * scale
            p = torch.softmax(x, -1)
            out[n, i] = (p @ vv).view(Hq, d)
            lse[n, i] = torch.logsumexp(x, -1).view(Hq)
            # a sum of d fp32 products; 8 more for the scaling, the exponential and its argument.
            # The 8-bit cache's queries are held to 2^-25 of their row's largest.
            big = (qq.abs() @ kk.abs()).amax(-1) + qq.abs().amax(-1) * kk.abs().sum(1).amax(-1)[:, None]
            ds = (d + 8) * 2.0 ** -24 * abs(scale) * big + 2.0 ** -22 * x.abs().amax(-1)
            spread = (p @ vv.abs())
            t = half * (p @ vv).abs() + spread * (half + 2 * ds + 2.0 ** -18)[..., None]
            tol[n, i] = t.view(Hq, d) + 2.0 ** -24
            ltol[n, i] = (ds + 2.0 ** -18).view(Hq) + lse[n, i].abs() * 2.0 ** -23
    return out, lse, tol, ltol


def assert_within(x, ref, tol, what):
    x = x.double().cpu()
    assert torch.equal(torch.isfinite(x), torch.isfinite(ref)), f"{what}: other infinities or NaN"
    fine = torch.isfinite(ref)
    assert torch.equal(x[~fine], ref[~fine]), f"{what}: infinities"
    over = (x - ref)[fine].abs() - tol.expand(ref.shape)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: {float(over.max()):.3e} over the tolerance, at {int(over.argmax())} of {over.numel()}"
