"""The rollout's key/value cache in NVFP4, rotary frequencies, and a layer's
attention over the cache on both sides of RL alignment.

[TRACE] "Le problème", "Résultats": the rollout keeps weights, activations
and the KV cache in FP4.  KVCache holds the pages and their decode scales; it
is written with binding.kv_cache_write, attended with
binding.attention_paged and read back with binding.kv_cache_read.
"""
import math

import torch

from . import binding as B
from . import workloads as W


class KVCache:
    """A paged NVFP4 key/value cache: codes [n_pages, n_heads, page_size, D / 2],
    scales [n_pages, n_heads, page_size, D / 16], decode scales g [n_heads].
    Wraps the given tensors; KVCache.empty allocates them.  The calls go by the
    tensors' addresses, so the attributes cannot be set: other tensors are
    another KVCache (values are changed in place, storage is not; a deep copy has
    its own)."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, g_k, g_v):
        codes, dev = k_codes.shape, k_codes.get_device()
        n_pages, n_heads, page_size, half = codes
        scales, heads = (n_pages, n_heads, page_size, half // 8), (n_heads,)
        u8, f32 = torch.uint8, torch.float32
        # written out: a cache may be wrapped around its tensors once per step
        if not (k_codes.dtype is u8 and v_codes.dtype is u8 and k_scales.dtype is u8 and v_scales.dtype is u8
                and g_k.dtype is f32 and g_v.dtype is f32
                and v_codes.shape == codes and k_scales.shape == scales and v_scales.shape == scales
                and g_k.shape == heads and g_v.shape == heads
                and v_codes.get_device() == dev and k_scales.get_device() == dev and v_scales.get_device() == dev
                and g_k.get_device() == dev and g_v.get_device() == dev
                and k_codes.is_contiguous() and v_codes.is_contiguous() and k_scales.is_contiguous()
                and v_scales.is_contiguous() and g_k.is_contiguous() and g_v.is_contiguous()):
            got = ", ".join(f"{n} {t.dtype} {tuple(t.shape)} on {t.device}" for n, t in (
                ("k_codes", k_codes), ("k_scales", k_scales), ("v_codes", v_codes), ("v_scales", v_scales),
                ("g_k", g_k), ("g_v", g_v)))
            raise ValueError(f"a cache needs contiguous uint8 codes {tuple(codes)}, uint8 scales {scales} and float32 "
                             f"decode scales {heads} on one device, got {got}")
        if g_k.requires_grad or g_v.requires_grad:
            raise ValueError("a cache's decode scales are fixed while its tokens are in use: pass detached tensors")
        a = self.__dict__
        a["n_pages"], a["n_heads"], a["page_size"], a["head_dim"] = n_pages, n_heads, page_size, 2 * half
        a["k_codes"], a["k_scales"], a["v_codes"], a["v_scales"] = k_codes, k_scales, v_codes, v_scales
        a["g_k"], a["g_v"] = g_k, g_v
        a["desc"] = B.kv_cache_desc(n_pages, page_size, n_heads, 2 * half, 0, k_codes.data_ptr(), k_scales.data_ptr(),
                                    v_codes.data_ptr(), v_scales.data_ptr(), g_k.data_ptr(), g_v.data_ptr())

    def __setattr__(self, name, value):
        raise AttributeError(f"a KVCache's {name} cannot be changed: make another KVCache")

    def __delattr__(self, name):
        raise AttributeError(f"a KVCache's {name} cannot be changed: make another KVCache")

    def __reduce__(self):                                # copies describe their own tensors
        return type(self), (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.g_k, self.g_v)

    @classmethod
    def empty(cls, n_pages, page_size, n_heads, head_dim, amax_k, amax_v, device="cuda"):
        """Pages of zeros for heads whose largest |k| and |v| are amax_k and
        amax_v (tensors [n_heads], or one number for all heads)."""
        def g(a):
            a = torch.as_tensor(a, dtype=torch.float32, device=device).expand(n_heads)
            return (a / 2688.0).contiguous()
        z = lambda d: torch.zeros((n_pages, n_heads, page_size, d), dtype=torch.uint8, device=device)
        return cls(z(head_dim // 2), z(head_dim // 16), z(head_dim // 2), z(head_dim // 16), g(amax_k), g(amax_v))


def rope_frequencies(rot_dim, theta=10000.0, scaling=None, factor=1.0, original_len=None, low=1.0, high=32.0,
                     device="cuda"):
    """Radians per position of each of the rot_dim / 2 pairs, float64, for
    binding.rope: theta ** (-2 f / rot_dim), changed for contexts `factor`
    times as long as `original_len`:
      scaling None       unchanged;
      "linear"           divided by factor (positions interpolated);
      "base"             theta * factor ** (rot_dim / (rot_dim - 2)), so that the
                         slowest pair is divided by factor and the fastest kept;
      "by_turns"         pairs that turn at most `low` times in original_len
                         positions divided by factor, those that turn at least
                         `high` times kept, those between mixed linearly in
                         their turns.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be a positive even number")
    if not factor > 0:
        raise ValueError("factor must be positive")
    f = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError('scaling "base" needs rot_dim >= 4')
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    freq = float(theta) ** (-2.0 * f / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_turns":
        if original_len is None or not high > low:
            raise ValueError('scaling "by_turns" needs original_len and low < high')
        keep = ((freq * original_len / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device)


class CachedAttention:
    """One layer's attention: BF16 projections (library matmuls), rotary
    positions, the paged NVFP4 cache and the attention over it.

    Rollout: keys and values are quantized into the cache as they are written
    and the new tokens attend over it.  Trainer: in a recorded layer its own
    queries attend over the rollout's cache, the values the rollout used
    ([TRACE] "Fonctionnement": the trainer reproduces them); elsewhere it
    quantizes its own keys and values on the same grid, with the rollout's
    decode scales, into a cache of its own.
    """

    def __init__(self, acfg: W.AttnConfig, w_qkv, w_o, lengths, device="cuda"):
        self.cfg, self.w_qkv, self.w_o = acfg, w_qkv, w_o
        self.dev = torch.device(device)
        self.lengths = [int(n) for n in lengths]
        self.T, self.longest = sum(self.lengths), max(self.lengths)
        pages = [-(-n // acfg.page) for n in self.lengths]
        self.n_pages, width = sum(pages), max(pages)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=self.dev)
        first = [sum(pages[:b]) for b in range(len(pages))]
        self.table = i32([[first[b] + j if j < pages[b] else -1 for j in range(width)] for b in range(len(pages))])
        self.off = i32([sum(self.lengths[:b]) for b in range(len(pages) + 1)])
        self.kv_len = i32(self.lengths)
        self.pos = torch.cat([torch.arange(n, device=self.dev) for n in self.lengths])
        self.freq = rope_frequencies(acfg.rot, acfg.theta, device=self.dev)
        self.cache = self.t_cache = None

    def project(self, x):
        """Rotated queries and keys, and values, of x [T, H]: [T, heads, dim] each."""
        c = self.cfg
        qkv = (x @ self.w_qkv.t()).view(self.T, c.heads_q + 2 * c.heads_k, c.dim)
        q, k = B.rope(qkv[:, :c.heads_q], qkv[:, c.heads_q:c.heads_q + c.heads_k], self.pos, self.freq,
                      interleaved=c.interleaved)
        return q, k, qkv[:, c.heads_q + c.heads_k:]

    def calibrate(self, x):
        """Sets each head's decode scales from x and allocates both sides' caches."""
        _, k, v = self.project(x)
        amax = [t.abs().amax(dim=(0, 2)).float() for t in (k, v)]
        c = self.cfg
        self.cache, self.t_cache = (KVCache.empty(self.n_pages, c.page, c.heads_k, c.dim, *amax, device=self.dev)
                                    for _ in range(2))

    def attend(self, q, cache):
        o = B.attention_paged(q, cache, self.off, self.kv_len, self.table, self.longest, window=self.cfg.window)
        return o.view(self.T, -1) @ self.w_o.t()

    def rollout(self, x):
        """The attention's output [T, H]; leaves keys and values in the cache."""
        q, k, v = self.project(x)
        B.kv_cache_write(self.cache, k, v, self.off, self.kv_len, self.table)
        return self.attend(q, self.cache)

    def trainer(self, x, replay):
        """The trainer's output [T, H]: over the rollout's cache (replay), or
        over its own keys and values on the same grid."""
        q, k, v = self.project(x)
        if replay:
            return self.attend(q, self.cache)
        B.kv_cache_write(self.t_cache, k, v, self.off, self.kv_len, self.table)
        return self.attend(q, self.t_cache)

    def kv_gap(self, x):
        """Relative distances of the trainer's own keys and values of x from
        those that the rollout cached, read back (a reported diagnostic)."""
        _, k, v = self.project(x)
        kr, vr = B.kv_cache_read(self.cache, self.off, self.table, self.T, out_dtype=B.OUT_F32)
        rel = lambda a, b: float(torch.linalg.vector_norm(a.float() - b) / torch.linalg.vector_norm(b).clamp_min(1e-30))
        return rel(k, kr), rel(v, vr)
