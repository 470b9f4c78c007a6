"""What the tests of the KV cache share: random caches and sequences, a 64-bit
torch form of the attention (any device; checked against the oracle on the
CPU) and the error bounds."""
import math

import numpy as np
import torch

from oracle import formats as F


def make_cache(n_pages, heads, page, dim, seed, device="cpu", spread=1.0, zero_scales=False):
    """Random codes and scales of a cache, as torch tensors."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8)
    t = {"k_codes": r(0, 256, n_pages, heads, page, dim // 2), "v_codes": r(0, 256, n_pages, heads, page, dim // 2),
         "k_scales": r(0x58, 0x7F, n_pages, heads, page, dim // 16),
         "v_scales": r(0 if zero_scales else 0x50, 0x7F, n_pages, heads, page, dim // 16),
         "g_k": spread * (0.5 + torch.rand(heads, generator=g)) / 600.0, "g_v": (0.5 + torch.rand(heads, generator=g)) / 600.0}
    return {n: x.to(device) for n, x in t.items()}


def oracle_cache(t):
    """The same cache as the oracle's arrays."""
    n = {name: x.cpu().numpy() for name, x in t.items()}
    return {"k_codes": F.unpack_nibbles(n["k_codes"]), "v_codes": F.unpack_nibbles(n["v_codes"]),
            "k_scales": n["k_scales"], "v_scales": n["v_scales"], "g_k": n["g_k"].astype(np.float64),
            "g_v": n["g_v"].astype(np.float64)}


def make_table(kv, page, n_pages, max_pages, seed):
    """Block table [n_seqs, max_pages] int32 of distinct shuffled pages, -1 behind each sequence's last."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in kv]
    assert sum(need) <= n_pages and max(need, default=0) <= max_pages
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(kv), max_pages), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))


def values64(t, name):
    """e2m1 * e4m3 * g of a whole cache side, float64 [pages, heads, page, D]."""
    dev = t["k_codes"].device
    level = torch.tensor(F.e2m1_value(np.arange(16)), dtype=torch.float64, device=dev)
    scale = torch.tensor(F.e4m3_value(np.arange(127)), dtype=torch.float64, device=dev)
    c = t[name + "_codes"]
    v = level[torch.stack([c & 15, c >> 4], -1).flatten(-2).long()]
    return v * scale[t[name + "_scales"].long()].repeat_interleave(16, -1) * t["g_" + name].double()[None, :, None, None]


def attention64(q, t, row_off, kv_len, table, scale, window=0):
    """out, lse, vabs, sabs, vsum as oracle.kvcache.attention gives them, in float64 torch."""
    dev, (rows, hq, D) = q.device, q.shape
    n_pages, hk, ps, _ = t["k_codes"].shape
    kd, vd = values64(t, "k"), values64(t, "v")
    f = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    out, vabs, vsum, sabs = f(rows, hq, D), f(rows, hq, D), f(rows, hq, D), f(rows, hq)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=dev)
    off, lens, tab = row_off.tolist(), kv_len.tolist(), table.cpu()
    for b, length in enumerate(lens):
        n = off[b + 1] - off[b]
        length = max(0, min(length, tab.shape[1] * ps))
        if n == 0 or length == 0:
            continue
        j = torch.arange(length)
        page = tab[b, j // ps].long()
        has = ((page >= 0) & (page < n_pages)).to(dev)
        page, at = page.clamp(0, n_pages - 1).to(dev), (j % ps).to(dev)
        k = kd[page, :, at].repeat_interleave(hq // hk, 1)
        v = vd[page, :, at].repeat_interleave(hq // hk, 1)
        for i0 in range(0, n, 256):
            i = torch.arange(i0, min(n, i0 + 256))
            pos = (lens[b] - n + i).to(dev)[:, None]
            see = (j.to(dev)[None] <= pos) & has[None]
            if window:
                see &= j.to(dev)[None] > pos - window
            rr = slice(off[b] + i0, off[b] + i0 + len(i))
            qq = q[rr].double()
            s = torch.einsum("nhd,lhd->nhl", qq, k) * scale
            s = s.masked_fill(~see[:, None], -math.inf)
            any_ = see.any(1)[:, None].expand(-1, hq)
            m = torch.where(any_, s.amax(-1), 0.0)
            e = torch.exp(s - m[..., None])
            l = torch.where(any_, e.sum(-1), 1.0)
            w = e / l[..., None]
            out[rr] = torch.einsum("nhl,lhd->nhd", w, v)
            vabs[rr] = torch.einsum("nhl,lhd->nhd", w, v.abs())
            vsum[rr] = torch.einsum("nl,lhd->nhd", see.double(), v.abs())
            lse[rr] = torch.where(any_, m + torch.log(l), -math.inf)
            a = torch.einsum("nhd,lhd->nhl", qq.abs(), k.abs()) * abs(scale)
            sabs[rr] = a.masked_fill(~see[:, None], 0.0).amax(-1)
    return out, lse, vabs, sabs, vsum


def attention_bounds(out, lse, vabs, sabs, vsum, dim):
    """Elementwise bounds on a kernel's out (BF16) and lse (FP32).

    A score is a sum of dim products of exact factors, each of at most dim
    additions rounded to 32 bits (2^-23 of the partial sum, truncation
    included): off by at most d = dim 2^-23 sabs, and by 2^-22 sabs more for
    its scaling.  A weight rounded to 16 bits is off by 2^-11 (FP16), its
    exponential by 2^-21, the average of the scores' errors by 2 d; all of
    that times the weighted |v|.  Sums of n weights in 32 bits add 2^-16 at
    most here.  FP16's steps do not shrink below 2^-24: with weights held at
    2^7 times their share of a maximum that some key attains, each is off by
    at most 2^-25 / 2^7 = 2^-32 of a sum that is at least that maximum's.  The
    result is rounded to BF16: 2^-8 of it."""
    d = sabs * (dim * 2.0 ** -23 + 2.0 ** -22)
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2.0 ** -15 + 2 * d[..., None]) * vabs * (1 + 2.0 ** -7) + \
        2.0 ** -32 * vsum * (1 + 2.0 ** -7) + 1e-30
    tol_lse = d + 2.0 ** -16 + 2.0 ** -22 * torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    return tol, tol_lse
