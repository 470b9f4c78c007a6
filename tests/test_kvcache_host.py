"""Refusals of the KV cache's entry points, on the host: no launch is made."""
import math

import pytest
import torch

from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B
from train_alignment_b200 import workloads as W

P = 1 << 20          # a stand-in for an aligned device address: no call below reaches the device


@pytest.fixture(scope="module")
def lib():
    from train_alignment_b200 import build
    build.build()
    return B.load()


def desc(**kw):
    d = dict(n_pages=8, page_size=16, n_heads=2, head_dim=128, k_codes=P, k_scales=P, v_codes=P, v_scales=P, g_k=P, g_v=P)
    d.update(kw)
    return B.kv_cache_desc(d["n_pages"], d["page_size"], d["n_heads"], d["head_dim"], 0,
                           *(d[n] or 0 for n in ("k_codes", "k_scales", "v_codes", "v_scales", "g_k", "g_v")))


BAD_CACHES = [dict(n_pages=-1), dict(n_pages=1 << 31), dict(page_size=0), dict(page_size=24), dict(page_size=1 << 17),
              dict(n_heads=0), dict(n_heads=2000), dict(head_dim=96), dict(head_dim=0), dict(n_pages=1 << 30, page_size=64), dict(k_codes=None), dict(v_scales=None),
              dict(g_k=None), dict(v_codes=P + 8)]


def write(l, cache=None, k=P, v=P, rows=4, ld_k=256, ld_v=256, off=P, kv=P, table=P, n=2, pages=3):
    return l.quads_kv_cache_write(cache if cache is not None else desc(), k, v, rows, ld_k, ld_v, off, kv, table, n, pages, None)


def read(l, cache=None, off=P, start=None, table=P, n=2, pages=3, rows=4, k=P, v=P, dt=0):
    return l.quads_kv_cache_read(cache if cache is not None else desc(), off, start, table, n, pages, rows, k, v, dt, None)


def attend(l, cache=None, q=P, rows=4, ld=1024, hq=8, off=P, kv=P, table=P, n=2, pages=3, mq=2, scale=0.1, window=0, out=P << 8,
           lse=None, ws=P, ws_bytes=1 << 40):
    return l.quads_attention_paged(q, rows, ld, hq, cache if cache is not None else desc(), off, kv, table, n, pages, mq, scale,
                                   window, out, lse, ws, ws_bytes, None)


def rope(l, q=P, ld_q=256, hq=2, k=P, ld_k=128, hk=1, T=4, dim=128, pos=P, freq=P, rot=128, oq=P, ldo_q=256, ok=P, ldo_k=128):
    return l.quads_rope(q, ld_q, hq, k, ld_k, hk, T, dim, pos, freq, rot, 0, 1.0, 0, oq, ldo_q, ok, ldo_k, None)


BAD = [(write, dict(rows=-1)), (write, dict(ld_k=250)), (write, dict(ld_v=128)), (write, dict(k=None)), (write, dict(kv=None)),
       (write, dict(v=P + 2)), (write, dict(n=-1)), (write, dict(n=70000)), (write, dict(off=None)), (write, dict(table=None)),
       (write, dict(pages=-1)),
       (read, dict(rows=-1)), (read, dict(dt=2)), (read, dict(k=None, v=None)), (read, dict(k=P + 16)), (read, dict(off=None)),
       (attend, dict(rows=1 << 31)), (attend, dict(hq=7)), (attend, dict(hq=0)), (attend, dict(hq=8192, ld=1 << 21)),
       (attend, dict(ld=1000)), (attend, dict(ld=1028)), (attend, dict(window=-1)), (attend, dict(mq=-1)),
       (attend, dict(scale=float("nan"))), (attend, dict(scale=float("inf"))), (attend, dict(q=None)), (attend, dict(out=None)),
       (attend, dict(kv=None)), (attend, dict(pages=1000, ws=None)), (attend, dict(pages=1000, ws_bytes=100)),
       (attend, dict(pages=1000, ws=P + 4)), (attend, dict(rows=100, mq=50, pages=1000, ws_bytes=100)),
       (attend, dict(n=60000, pages=2000000)), (attend, dict(q=P + 8)), (attend, dict(out=P + 8)),
       (attend, dict(pages=(1 << 27) - (1 << 12) + 1)), (attend, dict(out=P)), (attend, dict(rows=5, out=P + 2 * (4 * 1024 + 1016))), (attend, dict(out=P - 2 * 4 * 1024 + 16)),
       (rope, dict(T=-1)), (rope, dict(hq=0, hk=0)), (rope, dict(dim=120)), (rope, dict(dim=2048)), (rope, dict(rot=8)),
       (rope, dict(rot=144)), (rope, dict(ld_q=128)), (rope, dict(ldo_k=132)), (rope, dict(q=None)), (rope, dict(ok=None)),
       (rope, dict(pos=None)), (rope, dict(freq=None)), (rope, dict(oq=P + 8))]


@pytest.mark.parametrize("call,kw", BAD, ids=[f"{c.__name__}-{'-'.join(k)}" for c, k in BAD])
def test_bad_arguments(lib, call, kw):
    n = lib.quads_launch_count()
    assert call(lib, **kw) in (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED_SHAPE)
    assert lib.quads_last_error().decode() != "" and lib.quads_launch_count() == n


@pytest.mark.parametrize("kw", BAD_CACHES, ids=[str(k) for k in BAD_CACHES])
@pytest.mark.parametrize("call", [write, read, attend])
def test_bad_caches(lib, call, kw):
    assert call(lib, cache=desc(**kw)) in (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED_SHAPE)
    assert lib.quads_last_error().decode() != ""


@pytest.mark.parametrize("call,kw", [(write, dict(rows=0)), (write, dict(n=0)), (write, dict(pages=0)), (read, dict(rows=0)),
                                     (read, dict(n=0)), (attend, dict(rows=0)), (attend, dict(n=0)), (attend, dict(mq=0)),
                                     (rope, dict(T=0))])
def test_nothing_to_do(lib, call, kw):
    n = lib.quads_launch_count()
    assert call(lib, **kw) == B.OK and lib.quads_launch_count() == n


def test_cache_tensors_are_checked():
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)
    g = torch.ones(2)
    ok = [z(4, 2, 16, 64), z(4, 2, 16, 8), z(4, 2, 16, 64), z(4, 2, 16, 8), g, g]
    A.KVCache(*ok)
    for i, bad in ((1, z(4, 2, 16, 4)), (2, z(4, 2, 32, 64)), (3, z(4, 2, 16, 8).float()), (4, torch.ones(3)),
                   (5, torch.ones(2, dtype=torch.float64)), (0, z(4, 2, 64, 16).transpose(2, 3))):
        with pytest.raises(ValueError):
            A.KVCache(*[bad if j == i else t for j, t in enumerate(ok)])
    c = A.KVCache.empty(3, 32, 2, 64, 6.0, torch.tensor([1.0, 2.0]), device="cpu")
    assert c.k_codes.shape == (3, 2, 32, 32) and c.v_scales.shape == (3, 2, 32, 4)
    assert torch.equal(c.g_v, torch.tensor([1.0, 2.0]) / 2688)


def test_host_tensors_are_refused(lib):
    c = A.KVCache.empty(3, 32, 2, 64, 6.0, 6.0, device="cpu")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: B.kv_cache_write(c, x, x, i, i[:1], i.view(1, 2)), lambda: B.kv_cache_read(c, i, i.view(1, 2), 4),
                 lambda: B.attention_paged(x, c, i, i[:1], i.view(1, 2), 4),
                 lambda: B.rope(x, None, torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rope_frequencies():
    f = A.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and f[0] == 1.0 and math.isclose(f[16], 1e-2)
    assert torch.allclose(A.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu"), f / 4)
    b = A.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert b[0] == 1.0 and math.isclose(b[-1], f[-1] / 4, rel_tol=1e-12)
    t = A.rope_frequencies(64, scaling="by_turns", factor=4.0, original_len=4096, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(t[turns >= 32], f[turns >= 32]) and torch.allclose(t[turns <= 1], f[turns <= 1] / 4)
    for bad in (dict(rot_dim=7), dict(rot_dim=64, scaling="x"), dict(rot_dim=64, scaling="by_turns"),
                dict(rot_dim=64, factor=0.0), dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            A.rope_frequencies(device="cpu", **bad)


def test_sequence_lengths():
    for T, n in ((300, 3), (4096, 5), (7, 7), (1, 1)):
        lens = W.sequence_lengths(T, n)
        assert len(lens) == n and sum(lens) == T and all(x >= 0 for x in lens)
    assert len(set(W.sequence_lengths(4096, 5))) == 5
