"""Pins of the oracle's KV cache, attention and rotary positions on the CPU,
and of the 64-bit torch form that the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

from oracle import kvcache as K
from oracle import nvfp4 as Q
from tests import kvcache_ref as R


def _case(seed, heads=2, group=2, dim=64, page=16, kv=(5, 40, 0, 17), new=(2, 9, 0, 17)):
    t = R.make_cache(9, heads, page, dim, seed)
    q = torch.randn((sum(new), heads * group, dim), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    return t, q, R.offsets(new), torch.tensor(kv, dtype=torch.int32), R.make_table(kv, page, 9, 4, seed)


@pytest.mark.parametrize("window", [0, 1, 7])
def test_torch_form_equals_the_oracle(window):
    t, q, off, kv, table = _case(3)
    table[1, 1] = 99                                   # a page that the cache has not
    o = K.attention(q.double().numpy(), R.oracle_cache(t), off.numpy(), kv.numpy(), table.numpy(), 0.125, window)
    r = R.attention64(q, t, off, kv, table, 0.125, window)
    for a, b in zip(o, r):
        b = b.numpy()
        assert np.array_equal(np.isfinite(a), np.isfinite(b))
        np.testing.assert_allclose(a[np.isfinite(a)], b[np.isfinite(b)], rtol=1e-12, atol=1e-12)


def test_one_visible_token_gives_its_value():
    t, q, off, kv, table = _case(4)
    out, lse = K.attention(q.double().numpy(), R.oracle_cache(t), off.numpy(), kv.numpy(), table.numpy(), 0.3, 1)[:2]
    c = R.oracle_cache(t)
    for r, (b, pos) in enumerate(K.row_positions(off.numpy(), kv.numpy())):
        at = K.place(c, table.numpy(), b, pos)
        for h in range(4):
            np.testing.assert_allclose(out[r, h], K.token(c, "v", at, h // 2), rtol=1e-14)
            s = 0.3 * (q[r, h].double().numpy() @ K.token(c, "k", at, h // 2))
            assert abs(lse[r, h] - s) < 1e-12


def test_rows_that_see_nothing_are_zero():
    t, q, off, _, table = _case(5, kv=(5, 40, 0, 17), new=(2, 9, 0, 17))
    kv = torch.tensor([0, 4, 0, 17], dtype=torch.int32)    # more new rows than tokens: negative positions
    out, lse = K.attention(q.double().numpy(), R.oracle_cache(t), off.numpy(), kv.numpy(), table.numpy(), 0.1)[:2]
    assert not out[:7].any() and np.isneginf(lse[:7]).all() and np.isfinite(lse[7:]).all()


def test_write_then_read_is_the_quantizer():
    rng = np.random.default_rng(0)
    t, _, off, kv, table = _case(6, dim=64)
    c = R.oracle_cache(t)
    rows = int(off[-1])
    k = torch.tensor(rng.normal(size=(rows, 2, 64))).to(torch.bfloat16).double().numpy()
    v = torch.tensor(rng.normal(size=(rows, 2, 64))).to(torch.bfloat16).double().numpy()
    w = K.write(c, k, v, off.numpy(), kv.numpy(), table.numpy())
    start = kv.numpy() - np.diff(off.numpy())
    rk, rv = K.read(w, off.numpy(), table.numpy(), start)
    for x, y, g in ((k, rk, c["g_k"]), (v, rv, c["g_v"])):
        for h in range(2):
            codes, scales = Q.quantize_with_scale(x[:, h], g[h])
            np.testing.assert_array_equal(y[:, h], Q.dequant(codes, scales, g[h]))
    # the other places are as they were
    touched = {K.place(c, table.numpy(), b, p) for b, p in K.row_positions(off.numpy(), kv.numpy())}
    for page in range(9):
        for at in range(16):
            if (page, at) not in touched:
                assert np.array_equal(w["k_codes"][page, :, at], c["k_codes"][page, :, at])


def test_rope_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 3, 32))
    freq = 10000.0 ** (-np.arange(8) / 8)
    pos = np.array([0, 1, 2, 77, 10 ** 6])
    for inter in (False, True):
        y = K.rope(x, pos, freq, inter, 1.5)
        np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
        np.testing.assert_allclose(y[0, :, :16], 1.5 * x[0, :, :16])
        np.testing.assert_allclose(np.linalg.norm(y[..., :16], axis=-1), 1.5 * np.linalg.norm(x[..., :16], axis=-1))
        np.testing.assert_allclose(K.rope(y, pos, freq, inter, 1 / 1.5, inverse=True), x, atol=1e-12)
        # the inverse at m is the transpose: <R x, g> = <x, R^T g>
        g = rng.normal(size=x.shape)
        lhs, rhs = (y * g).sum(), (x * K.rope(g, pos, freq, inter, 1.5, inverse=True)).sum()
        assert math.isclose(lhs, rhs, rel_tol=1e-12)
    # a product of a query and a key depends on the distance alone
    a, b = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    dots = [(K.rope(a, [p], freq) * K.rope(b, [p + 11], freq)).sum() for p in (0, 5, 900)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)


def test_a_planted_mistake_is_seen():
    """The comparison that the GPU tests make rejects an attention that leaves
    out a row's own position, and one that forgets a head's scale."""
    t, q, off, kv, table = _case(7)
    ref = R.attention64(q, t, off, kv, table, 0.125)
    tol, _ = R.attention_bounds(*ref, 64)
    short = R.attention64(q, t, off, kv - 1, table, 0.125)[0]
    assert (((short - ref[0]).abs() > tol).any(-1)[ref[1].isfinite()]).float().mean() > 0.9
    wrong = {**t, "g_v": torch.ones(2) / 600}
    assert ((R.attention64(q, wrong, off, kv, table, 0.125)[0] - ref[0]).abs() > tol).any()
