"""The operators of attention over an NVFP4 key/value cache, measured: rotary
positions, the cache written and read back, and the attention that reads it.

run() makes a user's calls of this package where `own` is true, and computes
the same operators in elementary torch operations where it is false.

A sequence b has kv_len[b] tokens in the cache, of which the last
row_off[b + 1] - row_off[b] are this call's new tokens; its pages are named
by block_table[b].  Cached values are e2m1 * e4m3 * g: 4-bit codes, one
8-bit scale per 16 elements of a head, one FP32 scale per head.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases

def _rope(T, heads_q, heads_k, dim, rot, interleaved, inverse, far, stretch):
    return {"op": "rope", "T": T, "heads_q": heads_q, "heads_k": heads_k, "dim": dim, "rot": rot,
            "interleaved": interleaved, "inverse": inverse, "far": far, "stretch": stretch}


def _write(seqs, new, kv, heads_k, dim, page, out, spread):
    return {"op": "write", "seqs": seqs, "new": new, "kv": kv, "heads_k": heads_k, "dim": dim, "page": page,
            "out": out, "spread": spread}


def _read(seqs, kv, heads_k, dim, page, out, spread):
    return {"op": "read", "seqs": seqs, "new": kv, "kv": kv, "heads_k": heads_k, "dim": dim, "page": page,
            "out": out, "spread": spread}


def _attend(seqs, new, kv, heads_q, heads_k, dim, page, window, spread):
    return {"op": "attend", "seqs": seqs, "new": new, "kv": kv, "heads_q": heads_q, "heads_k": heads_k, "dim": dim,
            "page": page, "window": window, "spread": spread}


def listed():
    return [
        # the hidden 2048 rollout's step: one new token for each of 64 sequences
        {"name": "rope_step", **_rope(64, 16, 4, 128, 128, False, False, 4096, 1.0)},
        # the hidden 4096 prefill of 16384 tokens, positions of a lengthened context
        {"name": "rope_prefill", **_rope(16384, 32, 8, 128, 128, False, False, 1 << 20, 8.0)},
        # the trainer's gradient through pairs side by side, half of each head rotated
        {"name": "rope_grad", **_rope(4097, 16, 16, 64, 32, True, True, 32768, 1.0)},
        # the rollout's step writes one token for each of 64 sequences, and they are read back
        {"name": "write_step", **_write(64, 1, 4096, 4, 128, 16, "bf16", 1)},
        # prompts of eight sequences written, and read back as the trainer replays them
        {"name": "write_prefill", **_write(8, 3500, 4000, 8, 128, 64, "f32", 2)},
        # a few short answers read back
        {"name": "read_short", **_read(4, 300, 4, 64, 16, "f32", 3)},
        # whole contexts read back for the trainer
        {"name": "read_long", **_read(8, 8192, 8, 128, 32, "bf16", 4)},
        # one new token of one short sequence: latency
        {"name": "decode_one", **_attend(1, 1, 700, 16, 4, 128, 16, 0, 5)},
        # the hidden 2048 rollout's step: 64 sequences of different lengths
        {"name": "decode_batch", **_attend(64, 1, 4096, 16, 4, 128, 16, 0, 6)},
        # four long contexts, one new token each
        {"name": "decode_long", **_attend(4, 1, 65536, 32, 8, 128, 64, 0, 7)},
        # short and long pieces of prompts, a sliding window, a key head for each query head
        {"name": "chunk_window", **_attend(8, 256, 5000, 16, 16, 64, 16, 1024, 8)},
        # a piece of a prompt for two sequences of the hidden 4096 model
        {"name": "prefill", **_attend(2, 4096, 12000, 32, 8, 128, 32, 0, 9)},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    dim = rng.choice([64, 128])
    heads_k = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    spread = rng.randrange(1 << 20)
    if op == "rope":
        rot = rng.choice([dim, dim // 2, dim // 4])
        most = (16384 * 40 * 128) // ((group + 1) * heads_k * dim)
        return _rope(_log_int(rng, 1, min(16384, most)), group * heads_k, heads_k, dim, rot, rng.random() < 0.5,
                     rng.random() < 0.4, _log_int(rng, 1 << 8, 1 << 20), rng.choice([1.0, 4.0, 8.0]))
    seqs = _log_int(rng, 1, 64)
    if op == "write":
        new = _log_int(rng, 1, max(1, min(8192, 24000 * 8 // (seqs * heads_k))))
        return _write(seqs, new, new + _log_int(rng, 1, 512) - 1, heads_k, dim, page, rng.choice(["bf16", "f32"]),
                      spread)
    if op == "read":
        kv = _log_int(rng, 1, max(1, min(16384, 8 * 8192 * 8 // (seqs * heads_k))))
        return _read(seqs, kv, heads_k, dim, page, rng.choice(["bf16", "f32"]), spread)
    kv = _log_int(rng, 1, max(1, min(65536, 4 * 65536 * 8 // (seqs * heads_k))))
    heads_q = group * heads_k
    new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, min(kv, 4096, (1 << 30) // (seqs * kv * heads_q))))
    return _attend(seqs, new, kv, heads_q, heads_k, dim, page, rng.choice([0, 0, 128, 1000]), spread)


def _lengths(case):
    """New and total tokens of each sequence: ragged, the first as long as the case says."""
    rng = random.Random(case["spread"])
    same = case["op"] == "read"
    new, kv = [], []
    for b in range(case["seqs"]):
        n = case["new"] if b == 0 else rng.randint(1, case["new"])
        t = case["kv"] if b == 0 else rng.randint(min(case["kv"], max(n, case["kv"] // 8)), case["kv"])
        new.append(t if same else n)
        kv.append(t)
    return new, kv


# --------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "rope":
        T, D = case["T"], case["dim"]
        hq, hk, half = case["heads_q"], case["heads_k"], case["rot"] // 2
        # q and k as a projection of the hidden state leaves them: slices of one row per token
        qk = _normal((T, (hq + hk) * D), g)
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        turns = freq * case["far"] / (2 * math.pi)
        # slow frequencies are stretched to the longer context, fast ones kept, those between mixed
        mix = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        freq = freq * (mix + (1.0 - mix) / case["stretch"])
        return {"case": case, "q": qk[:, :hq * D].view(T, hq, D), "k": qk[:, hq * D:].view(T, hk, D),
                "pos": torch.randint(0, case["far"], (T,), generator=g, device=DEV), "freq": freq,
                "mscale": 0.1 * math.log(case["stretch"]) + 1.0}
    new, kv = _lengths(case)
    B, ps, D, hk = case["seqs"], case["page"], case["dim"], case["heads_k"]
    pages = [-(-n // ps) for n in kv]
    width = max(pages)
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(B)], device=DEV)
    count = torch.tensor(pages, device=DEV)
    j = torch.arange(width, device=DEV)
    table = torch.where(j[None] < count[:, None], order[(first[:, None] + j[None]).clamp(max=n_pages - 1)], -1)
    off = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    state = {"case": case, "row_off": off, "kv_len": torch.tensor(kv, dtype=torch.int32, device=DEV),
             "table": table.to(torch.int32).contiguous(), "rows": sum(new), "longest": max(new), "longest_kv": max(kv)}

    def cache_of(spread):
        # codes and scales as normal values leave them under a head's calibrated scale
        z = 5.0 * spread / 2688.0
        pick = torch.tensor([0, 1, 1, 2, 2, 3, 3, 4, 4, 4, 5, 5, 5, 6, 6, 7], dtype=torch.uint8, device=DEV)
        pick = torch.cat([pick, pick + 8])
        nib = pick[torch.randint(0, 32, (n_pages, hk, ps, D), generator=g, device=DEV, dtype=torch.uint8).int()]
        return ((nib[..., 0::2] | (nib[..., 1::2] << 4)).contiguous(),
                torch.randint(0x68, 0x7A, (n_pages, hk, ps, D // 16), generator=g, device=DEV, dtype=torch.uint8),
                (z * (0.7 + 0.6 * torch.rand(hk, generator=g, device=DEV))).float())

    state["k_codes"], state["k_scales"], state["g_k"] = cache_of(1.0)
    state["v_codes"], state["v_scales"], state["g_v"] = cache_of(0.8)
    if case["op"] == "write":
        rows = state["rows"]
        kvp = torch.randn((rows, 2, hk, D), generator=g, device=DEV)
        # keys with a few large channels, as they come; a head's calibrated range falls a little short of some
        kvp[:, 0, :, ::29] *= 6.0
        kvp = kvp.to(torch.bfloat16)
        state["k"], state["v"] = kvp[:, 0], kvp[:, 1]
        state["g_k"] = (kvp[:, 0].float().abs().amax(dim=(0, 2)).clamp(min=1.0) * 0.95 / 2688.0).contiguous()
        state["g_v"] = (kvp[:, 1].float().abs().amax(dim=(0, 2)).clamp(min=1.0) * 0.95 / 2688.0).contiguous()
    if case["op"] in ("write", "read"):
        state["start"] = state["kv_len"] - (off[1:] - off[:-1])
    if case["op"] == "attend":
        state["q"] = _normal((state["rows"], case["heads_q"], D), g)
        state["scale"] = D ** -0.5
    return state


# ----------------------------------------------- what the framework is asked

def _run_own(s):
    from train_alignment_b200 import attention as A
    from train_alignment_b200 import binding as B
    case = s["case"]
    if case["op"] == "rope":
        call = B.rope_backward if case["inverse"] else B.rope
        return call(s["q"], s["k"], s["pos"], s["freq"], interleaved=case["interleaved"], mscale=s["mscale"])
    cache = A.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["g_k"], s["g_v"])
    if case["op"] == "attend":
        return B.attention_paged(s["q"], cache, s["row_off"], s["kv_len"], s["table"], s["longest"],
                                 scale=s["scale"], window=case["window"])
    if case["op"] == "write":
        B.kv_cache_write(cache, s["k"], s["v"], s["row_off"], s["kv_len"], s["table"])
    return B.kv_cache_read(cache, s["row_off"], s["table"], s["rows"], start=s["start"],
                           out_dtype=B.OUT_F32 if case["out"] == "f32" else B.OUT_BF16)


# ----------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    x = x.float()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1).to(torch.bfloat16)


def _e4m3_table(dtype):
    c = torch.arange(128, device=DEV)
    e, m = c // 8, (c % 8).to(dtype)
    return torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).to(dtype)))


def _values(codes, scales, g, dtype=torch.float32):
    """e2m1 * e4m3 * g of packed codes [..., heads, D / 2] and scales [..., heads, D / 16]."""
    mag = torch.tensor(E2M1, dtype=dtype, device=DEV)
    lut = torch.cat([mag, -mag])
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = lut[nib.int()] * _e4m3_table(dtype)[scales.int()].repeat_interleave(16, -1)
    return v * g[:, None].to(dtype)


def _rows(s):
    """Sequence and position in the cache of each new row."""
    t = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(s["row_off"].long(), t, right=True) - 1
    first = s["kv_len"] - (s["row_off"][1:] - s["row_off"][:-1])
    return b, t - s["row_off"][b], first[b] + t - s["row_off"][b]


def _slots(s):
    b, _, pos = _rows(s)
    return s["table"][b, (pos // s["case"]["page"]).long()].long(), (pos % s["case"]["page"]).long()


def _quantise(x, g):
    """Packed codes and scale bytes of x [rows, heads, D] with a scale per head,
    each product and quotient rounded to 32 bits as the format has it."""
    r, h, d = x.shape
    x = x.float().view(r, h, d // 16, 16)
    g = g.view(1, h, 1)
    t = (x.abs().amax(-1) / (6.0 * g)).clamp(max=448.0)
    s = t.to(torch.float8_e4m3fn).view(torch.uint8)
    big = _e4m3_table(torch.float32)[s.int()] * g
    y = x * torch.where(big > 0, 1.0 / big, 0.0)[..., None]
    m = y.abs()
    # nearest level, ties to the even code
    c = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    c = (c + 8 * torch.signbit(x)).to(torch.uint8).view(r, h, d)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        angle = s["pos"].double()[:, None] * s["freq"][None]
        cos = (torch.cos(angle) * s["mscale"]).float()[:, None]
        sin = (torch.sin(angle) * s["mscale"]).float()[:, None]
        sin = -sin if case["inverse"] else sin
        return _rotate(s["q"], cos, sin, case["interleaved"]), _rotate(s["k"], cos, sin, case["interleaved"])
    if case["op"] == "attend":
        return _attention(s, torch.float32).to(torch.bfloat16)
    page, at = _slots(s)
    if case["op"] == "write":
        for_k, for_v = _quantise(s["k"], s["g_k"]), _quantise(s["v"], s["g_v"])
        s["k_codes"][page, :, at], s["k_scales"][page, :, at] = for_k
        s["v_codes"][page, :, at], s["v_scales"][page, :, at] = for_v
    out = torch.float32 if case["out"] == "f32" else torch.bfloat16
    return (_values(s["k_codes"][page, :, at], s["k_scales"][page, :, at], s["g_k"]).to(out),
            _values(s["v_codes"][page, :, at], s["v_scales"][page, :, at], s["g_v"]).to(out))


def _attention(s, dtype):
    """Softmax attention of every new row over its sequence, padded to the longest."""
    case = s["case"]
    B, hq, hk, D, ps = case["seqs"], case["heads_q"], case["heads_k"], case["dim"], case["page"]
    L, N = s["longest_kv"], s["longest"]
    b, i, pos = _rows(s)
    q = torch.zeros((B, N, hk, hq // hk, D), dtype=dtype, device=DEV)
    q[b, i] = s["q"].to(dtype).view(-1, hk, hq // hk, D)
    p = torch.zeros((B, N), dtype=torch.int64, device=DEV)
    p[b, i] = pos.long()
    j = torch.arange(L, device=DEV)
    page, at = s["table"][:, j // ps].clamp(min=0).long(), (j % ps).expand(B, L)
    k = _values(s["k_codes"][page, :, at], s["k_scales"][page, :, at], s["g_k"], dtype)
    v = _values(s["v_codes"][page, :, at], s["v_scales"][page, :, at], s["g_v"], dtype)
    seen = (j <= p[..., None]) & (j < s["kv_len"][:, None, None])
    if case["window"]:
        seen &= j > p[..., None] - case["window"]
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hk, -1, D), k.permute(0, 2, 3, 1)) * s["scale"]
    x = x.view(B, hk, hq // hk, N, L).masked_fill_(~seen[:, None, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hk, -1, L), v.transpose(1, 2)).view(B, hk, hq // hk, N, D)
    return o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, hq, D)


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------ what it cannot do without

def work(case):
    D = case["dim"]
    if case["op"] == "rope":
        n = case["T"] * (case["heads_q"] + case["heads_k"])
        return {"bytes": n * D * 4 + case["T"] * 8 + case["rot"] * 4, "flops": n * case["rot"] * 3}
    new, kv = _lengths(case)
    row = 2 * case["heads_k"] * D                      # elements of a token's keys and values
    packed = row // 2 + row // 16
    if case["op"] == "attend":
        w, pairs, need = case["window"], 0, 0
        for n, t in zip(new, kv):
            lens = [min(t - n + i + 1, w) if w else t - n + i + 1 for i in range(n)]
            pairs += sum(lens)
            need += min(t, n - 1 + w) if w else t
        return {"bytes": sum(new) * case["heads_q"] * D * 4 + need * packed, "flops": 4 * D * case["heads_q"] * pairs}
    out = row * (4 if case["out"] == "f32" else 2)
    given = row * 2 if case["op"] == "write" else 0
    return {"bytes": sum(new) * (given + packed + out), "flops": sum(new) * row * (6 if given else 2)}


# ----------------------------------------------------- the definition in 64 bits

def _exact_quantised(x, g):
    """The values that x stands for in the cache: the format's own roundings of
    each step to 32 bits, the arithmetic between them in 64."""
    r, h, d = x.shape
    x = x.double().reshape(r, h, d // 16, 16)
    g = g.double().view(1, h, 1)
    t = ((x.abs().amax(-1)) / (6.0 * g).float().double()).float().double().clamp(max=448.0)
    # E4M3: three bits behind the leading one, steps of 2^-9 below 2^-6, ties to even
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    sv = torch.round(t / step) * step
    big = (sv * g).float().double()
    inv = torch.where(big > 0, (1.0 / big).float().double(), 0.0)
    y = (x * inv[..., None]).float().double().abs().clamp(max=6.0)
    # E2M1: one bit behind the leading one, steps of 1/2 below 2, ties to even
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=1.0))) - 1)
    q = torch.round(y / step) * step
    return (torch.copysign(q, x) * sv[..., None] * g[..., None]).reshape(r, h, d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        half, sign = case["rot"] // 2, -1.0 if case["inverse"] else 1.0
        turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=DEV),
                           sign * s["pos"].double()[:, None] * s["freq"])[:, None]
        done = []
        for x in (s["q"].double(), s["k"].double()):
            part = x[..., :2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            part = part if case["interleaved"] else part.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            y = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            done.append(torch.cat([y, x[..., 2 * half:]], -1))
        return tuple(done)
    if case["op"] == "write":
        return _exact_quantised(s["k"], s["g_k"]), _exact_quantised(s["v"], s["g_v"])
    new, kv = _lengths(case)
    ps, D, hk = case["page"], case["dim"], case["heads_k"]
    level = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    scale_of = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()

    def cached(name, b, lo, hi):
        """[hi - lo, heads, D] values of positions lo .. hi - 1 of sequence b, page after page."""
        pages = s["table"][b, lo // ps:-(-hi // ps)].long()
        c, z = s[name + "_codes"][pages], s[name + "_scales"][pages]
        val = torch.empty(c.shape[:-1] + (D,), dtype=torch.float64, device=DEV)
        val[..., 0::2], val[..., 1::2] = level[(c & 15).long()], level[(c >> 4).long()]
        val = (val.unflatten(-1, (D // 16, 16)) * scale_of[z.long()][..., None]).flatten(-2)
        val = val * s["g_" + name].double()[None, :, None, None]
        val = val.transpose(1, 2).reshape(-1, hk, D)
        return val[lo - lo // ps * ps:hi - lo // ps * ps]

    if case["op"] == "read":
        return (torch.cat([cached("k", b, 0, kv[b]) for b in range(len(kv))]),
                torch.cat([cached("v", b, 0, kv[b]) for b in range(len(kv))]))
    if work(case)["flops"] > 4e12:
        return None
    G, w, outs, row = case["heads_q"] // hk, case["window"], [], 0
    for n, t in zip(new, kv):
        b = len(outs)
        lo = max(0, t - n + 1 - w) if w else 0
        k, v = cached("k", b, lo, t), cached("v", b, lo, t)
        q = s["q"][row:row + n].double()
        row += n
        part = torch.empty(n, case["heads_q"], D, dtype=torch.float64, device=DEV)
        for h in range(case["heads_q"]):
            for i0 in range(0, n, 1024):
                at = torch.arange(t - n + i0, t - n + min(n, i0 + 1024), device=DEV)[:, None]
                j = torch.arange(lo, t, device=DEV)[None]
                hide = (j > at) | (j <= at - w) if w else j > at
                x = (q[i0:i0 + 1024, h] @ k[:, h // G].T * s["scale"]).masked_fill(hide, -math.inf)
                part[i0:i0 + 1024, h] = torch.softmax(x, -1) @ v[:, h // G]
        outs.append(part)
    return torch.cat(outs)
