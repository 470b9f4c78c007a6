"""The paged NVFP4 KV cache, the attention over it and rotary positions on the
GPU, against the oracle and against 64-bit torch."""
import math

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kvcache as K
from tests import kvcache_ref as R
from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16).to(DEV)


def _cache(t):
    return A.KVCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], t["g_k"], t["g_v"])


# -------------------------------------------------------------------- rope


def _check_rope(got, x, pos, freq, inter, m, inverse=False):
    xn = x.double().cpu().numpy()
    ref = K.rope(xn, pos.cpu().numpy(), freq.cpu().numpy(), inter, m, inverse)
    half = len(freq)
    mag = np.abs(xn).copy()
    a, b = (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2]) if inter else (np.s_[..., :half], np.s_[..., half:2 * half])
    mag[a] = mag[b] = np.abs(xn[a]) + np.abs(xn[b])
    # half a BF16 step, and 2^-20 for cos and sin of an angle rounded to 32 bits and the products
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * m * mag + 1e-30
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()
    np.testing.assert_array_equal(got[..., 2 * half:].cpu().float().numpy(), x[..., 2 * half:].cpu().float().numpy())


@pytest.mark.parametrize("T,hq,hk,dim,rot", [(1, 1, 1, 16, 16), (3, 5, 1, 64, 32), (257, 4, 4, 128, 128), (64, 16, 4, 128, 64),
                                             (1000, 3, 0, 96, 48), (40, 2, 2, 256, 256), (33, 1, 1, 1024, 1024),
                                             (2500, 32, 8, 128, 128)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope(cuda_lib, T, hq, hk, dim, rot, inter):
    q, k = _randn((T, hq, dim), 1), (_randn((T, hk, dim), 2) if hk else None)
    pos = torch.randint(0, 1 << 22, (T,), generator=torch.Generator().manual_seed(3)).to(DEV)
    pos[0] = 0
    freq = A.rope_frequencies(rot, device=DEV)
    for call, inverse in ((B.rope, False), (B.rope_backward, True)):
        oq, ok = call(q, k, pos, freq, interleaved=inter, mscale=1.25)
        _check_rope(oq, q, pos, freq, inter, 1.25, inverse)
        if hk:
            _check_rope(ok, k, pos, freq, inter, 1.25, inverse)
        else:
            assert ok is None


def test_rope_strided_and_in_place(cuda_lib):
    T, hq, hk, dim = 77, 6, 2, 64
    buf = _randn((T, (hq + 2 * hk) * dim), 5)
    keep = buf.clone()
    q, k = buf[:, :hq * dim].view(T, hq, dim), buf[:, hq * dim:(hq + hk) * dim].view(T, hk, dim)
    pos = torch.arange(T, device=DEV) * 1000
    freq = A.rope_frequencies(32, device=DEV)
    want = B.rope(q, k, pos, freq)
    B.rope(q, k, pos, freq, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, (hq + hk) * dim:], keep[:, (hq + hk) * dim:])


def test_rope_gradient_against_differences(cuda_lib):
    """The backward's product with a direction is the difference quotient of
    the forward (which is linear, so a wide step has no error of its own)."""
    T, h, dim = 31, 3, 64
    freq = A.rope_frequencies(64, scaling="by_turns", factor=4.0, original_len=4096, device=DEV)
    pos = torch.arange(T, device=DEV) * 411
    x, d, g = (_randn((T, h, dim), s) for s in (7, 8, 9))
    for inter in (False, True):
        gx = B.rope_backward(g, None, pos, freq, interleaved=inter, mscale=1.1)[0].double().cpu().numpy()
        f = lambda z: K.rope(z, pos.cpu().numpy(), freq.cpu().numpy(), inter, 1.1)
        xn, dn, gn = (z.double().cpu().numpy() for z in (x, d, g))
        quotient = ((f(xn + dn) - f(xn - dn)) / 2 * gn).sum((1, 2))
        # every product of gx is off by at most 2^-8 of it (the rounding to BF16), and a little for the sums
        bound = (2.0 ** -8 * np.abs(gx * dn) + 2.0 ** -19 * np.abs(dn)).sum((1, 2))
        assert (np.abs((gx * dn).sum((1, 2)) - quotient) <= bound * 1.01 + 2.0 ** -18 * np.abs(gn).sum((1, 2))).all()


# -------------------------------------------------------- writing and reading


@pytest.mark.parametrize("heads,dim,page,new,kv", [
    (1, 64, 16, [1], [1]), (2, 128, 16, [1] * 5, [1, 16, 17, 32, 100]), (4, 64, 48, [0, 7, 100, 0, 1], [3, 7, 130, 0, 49]),
    (8, 128, 64, [33, 250], [40, 250])])
def test_write_and_read(cuda_lib, heads, dim, page, new, kv):
    n_pages = sum(-(-n // page) for n in kv) + 3
    t = R.make_cache(n_pages, heads, page, dim, 1, DEV)
    rows = sum(new)
    k, v = _randn((rows, heads, dim), 2, 3.0), _randn((rows, heads, dim), 3)
    k[rows // 2] = 0.0                                     # a block of zeros
    v[-1] *= 2.0 ** -20                                    # blocks whose scale rounds to zero
    # some values above the calibrated range
    t["g_k"] = (k.float().abs().amax((0, 2)).clamp(min=0.5) * 0.8 / 2688).contiguous()
    t["g_v"] = (v.float().abs().amax((0, 2)).clamp(min=0.5) / 2688).contiguous()
    off, lens, table = R.offsets(new), torch.tensor(kv, dtype=torch.int32), R.make_table(kv, page, n_pages, 12, 4)
    want = K.write(R.oracle_cache(t), k.double().cpu().numpy(), v.double().cpu().numpy(), off.numpy(), lens.numpy(),
                   table.numpy())
    cache = _cache(t)
    B.kv_cache_write(cache, k, v, off.to(DEV), lens.to(DEV), table.to(DEV))
    for name in ("k", "v"):
        np.testing.assert_array_equal(F.unpack_nibbles(t[name + "_codes"].cpu().numpy()), want[name + "_codes"])
        np.testing.assert_array_equal(t[name + "_scales"].cpu().numpy(), want[name + "_scales"])
    # read whole sequences back, and the new tokens alone, in both types
    start = lens - (off[1:] - off[:-1])
    for roff, st in ((R.offsets(kv), None), (off, start)):
        n = int(roff[-1])
        ref = K.read(want, roff.numpy(), table.numpy(), None if st is None else st.numpy())
        for dt in (B.OUT_F32, B.OUT_BF16):
            got = B.kv_cache_read(cache, roff.to(DEV), table.to(DEV), n, start=None if st is None else st.to(DEV),
                                  out_dtype=dt)
            for g, r in zip(got, ref):
                r = F.f32(r) if dt == B.OUT_F32 else F.bf16_rne(F.f32(r).astype(np.float32))
                np.testing.assert_array_equal(g.double().cpu().numpy(), r)


@pytest.mark.parametrize("lead", [0, 8, 16])
def test_write_from_wider_rows(cuda_lib, lead):
    """k and v as slices of a projection's rows, at 16- and 32-byte offsets."""
    heads, dim, rows = 4, 64, 70
    wide = _randn((rows, lead + 2 * heads * dim + 24), 1)
    k = wide[:, lead:lead + heads * dim].view(rows, heads, dim)
    v = wide[:, lead + heads * dim:lead + 2 * heads * dim].view(rows, heads, dim)
    off, kv, table = R.offsets([50, 20]).to(DEV), torch.tensor([50, 33], dtype=torch.int32, device=DEV), \
        R.make_table([50, 33], 16, 9, 4, 2).to(DEV)
    caches = [A.KVCache.empty(9, 16, heads, dim, 3.0, 3.0, DEV) for _ in range(2)]
    B.kv_cache_write(caches[0], k, v, off, kv, table)
    B.kv_cache_write(caches[1], k.contiguous(), v.contiguous(), off, kv, table)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)) and getattr(caches[0], n).any()


def test_write_and_read_leave_the_rest(cuda_lib):
    """Rows behind the last sequence, negative positions, positions without a
    page: nothing else is written; reading gives zeros without a page and
    leaves rows of no sequence."""
    heads, dim, page = 2, 64, 16
    t = R.make_cache(6, heads, page, dim, 5, DEV)
    cache = _cache(t)
    before = {n: x.clone() for n, x in t.items()}
    k, v = _randn((40, heads, dim), 6), _randn((40, heads, dim), 7)
    off = torch.tensor([0, 5, 5, 25, 30], dtype=torch.int32, device=DEV)
    kv = torch.tensor([2, 9, 200, 30], dtype=torch.int32, device=DEV)       # 3 rows before position 0; past the table
    table = torch.tensor([[0, -1], [1, 2], [3, 4], [-7, 6]], dtype=torch.int32, device=DEV)
    B.kv_cache_write(cache, k, v, off, kv, table)
    diff = (t["k_codes"] != before["k_codes"]).any(-1).any(1).nonzero().tolist()
    assert {tuple(x) for x in diff} <= {(0, 0), (0, 1)} and diff
    roff = torch.tensor([0, 5, 5, 12, 20], dtype=torch.int32, device=DEV)
    st = torch.tensor([14, 0, 30, -3], dtype=torch.int32, device=DEV)
    ko = torch.full((24, heads, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    vo = torch.full_like(ko, 9.0)
    B.kv_cache_read(cache, roff, table, 24, start=st, k_out=ko, v_out=vo)
    ref = K.read(R.oracle_cache(t), roff.cpu().numpy(), table.cpu().numpy(), st.cpu().numpy())
    np.testing.assert_array_equal(ko[:20].double().cpu().numpy(), F.bf16_rne(F.f32(ref[0]).astype(np.float32)))
    np.testing.assert_array_equal(vo[:20].double().cpu().numpy(), F.bf16_rne(F.f32(ref[1]).astype(np.float32)))
    assert (ko[20:] == 7.0).all() and (vo[20:] == 9.0).all() and not ko[2:5].any() and not ko[12:20].any()


# ---------------------------------------------------------------- attention


def _attend(heads, group, dim, page, new, kv, window=0, seed=1, extra=0, absent=(), garbage=False, spread=1.0, scale=None,
            q=None):
    """One call checked against 64 bits: out, lse, the rows behind the last sequence."""
    n_pages = sum(-(-max(n, 0) // page) for n in kv) + 2
    width = max([-(-max(n, 0) // page) for n in kv] + [1])
    t = R.make_cache(n_pages, heads, page, dim, seed, DEV, spread)
    off, lens = R.offsets(new), torch.tensor(kv, dtype=torch.int32)
    table = R.make_table(kv, page, n_pages, width, seed + 1)
    rows, hq = sum(new), heads * group
    if q is None:
        q = _randn((rows + extra, hq, dim), seed + 2)
    scale = dim ** -0.5 if scale is None else scale
    for b, j in absent:
        table[b, j] = (-1, n_pages, 1 << 30)[(b + j) % 3]
    ref = R.attention64(q[:rows], t, off.to(DEV), lens.to(DEV), table, scale, window)
    if garbage:
        # bytes of unwritten places: NaN patterns, behind each sequence and in the pages of none
        used = torch.zeros((n_pages, page), dtype=torch.bool)
        for b, n in enumerate(kv):
            for p in range(max(n, 0)):
                pg = int(table[b, p // page])
                if 0 <= pg < n_pages:
                    used[pg, p % page] = True
        free = (~used).to(DEV)[:, None, :, None]
        for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
            t[name].copy_(torch.where(free, torch.full_like(t[name], 0xFF), t[name]))
    out = torch.full((rows + extra, hq, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows + extra, hq), 5.0, dtype=torch.float32, device=DEV)
    B.attention_paged(q, _cache(t), off.to(DEV), lens.to(DEV), table.to(DEV), max(new), scale=scale, window=window, out=out,
                      lse=lse)
    assert B.device_status() == B.OK
    assert (out[rows:] == 3.0).all() and (lse[rows:] == 5.0).all()
    tol, tol_lse = R.attention_bounds(*ref, dim)
    got, got_lse = out[:rows].double(), lse[:rows].double()
    assert torch.equal(torch.isneginf(got_lse), torch.isneginf(ref[1])) and not got_lse.isnan().any()
    empty = torch.isneginf(ref[1])
    assert not got[empty].any()
    over = (got - ref[0]).abs() - tol
    assert not got.isnan().any() and (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()}, worst {over.max()}"
    dl = (got_lse - ref[1])[~empty].abs() - tol_lse[~empty]
    assert (dl <= 0).all(), dl.max()
    return out, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (4, 8), (1, 16), (2, 3), (3, 5), (1, 7), (2, 12)])
def test_single_tokens(cuda_lib, dim, heads, group):
    _attend(heads, group, dim, 16, [1] * 6, [1, 2, 16, 17, 333, 1000], seed=10 + group, extra=2, garbage=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 128, 1024])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_pages_and_windows(cuda_lib, dim, page, window):
    _attend(2, 4, dim, page, [1, 1, 1], [200, 700, 77], window, seed=20, garbage=True)
    _attend(2, 4, dim, page, [40, 1, 130], [200, 700, 130], window, seed=21, garbage=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new,kv", [
    (1, 1, [2], [2]), (2, 1, [129], [129]), (2, 4, [64, 65, 3], [64, 200, 1000]), (1, 8, [300], [777]),
    (4, 2, [1, 0, 17, 0, 250], [900, 0, 17, 40, 251]), (1, 3, [85, 86, 171], [85, 500, 171]), (1, 40, [5, 9], [300, 9]),
    (1, 300, [2, 1], [129, 128])])
def test_chunks(cuda_lib, dim, heads, group, new, kv):
    _attend(heads, group, dim, 32, new, kv, seed=30 + group, extra=3, garbage=True)
    _attend(heads, group, dim, 16, new, kv, window=90, seed=31 + group, garbage=True)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new,kv", [
    (2, 4, [3, 8, 12, 1, 0, 5], [300, 2000, 1100, 1500, 40, 5]), (1, 16, [3, 1, 2], [4000, 1100, 1025]),
    (1, 1, [48, 17, 33], [48, 900, 2000]), (3, 6, [8, 3], [8, 1300]), (1, 48, [1, 0, 1], [2100, 0, 700]),
    (2, 8, [8, 0, 7, 1], [3000, 0, 1100, 40]), (1, 64, [1, 1], [5000, 17]),
    (4, 4, [16, 9] + [1, 0, 3] * 13, [1500, 300] + [30, 0, 200] * 13)])
def test_rows_in_groups(cuda_lib, dim, heads, group, new, kv):
    """17 to 64 rows of a key head: several units, of which a sequence may have fewer."""
    _attend(heads, group, dim, 16, new, kv, seed=36, extra=1, garbage=True)
    _attend(heads, group, dim, 48, new, kv, window=130, seed=37, garbage=True)


@pytest.mark.parametrize("heads,n,longest", [(1, 200, 1500), (4, 200, 1500), (8, 129, 1500), (4, 200, 1000)])
def test_many_sequences(cuda_lib, heads, n, longest):
    """More sequences than one scan takes; units by themselves and by the CTA that begins them; sequences without rows."""
    kv = [1 + (37 * b) % longest for b in range(n)]
    new = [0 if b % 7 == 3 else 1 + b % 3 for b in range(n)]
    _attend(heads, 4, 64, 16, new, [max(k, m) for k, m in zip(kv, new)], seed=38)


@pytest.mark.parametrize("new", [[1, 1], [12, 3], [200, 60]])
def test_no_pages(cuda_lib, new):
    """A cache without pages, a table without columns, a table that ends before the sequence does."""
    for dim in (64, 128):
        t = R.make_cache(4, 2, 16, dim, 1, DEV)
        none = {n: (x[:0].contiguous() if x.dim() == 4 else x) for n, x in t.items()}
        off, lens = R.offsets(new).to(DEV), torch.tensor([300, 70], dtype=torch.int32, device=DEV)
        rows = sum(new)
        q = _randn((rows, 8, dim), 2)
        for cache, table in ((none, torch.zeros((2, 30), dtype=torch.int32)), (t, torch.zeros((2, 0), dtype=torch.int32)),
                             (none, torch.zeros((2, 0), dtype=torch.int32))):
            out, lse = torch.full_like(q, 4.0), torch.zeros((rows, 8), device=DEV)
            B.attention_paged(q, _cache(cache), off, lens, table.to(DEV), max(new), out=out, lse=lse)
            assert not out.any() and torch.isneginf(lse).all()
            k, v = B.kv_cache_read(_cache(cache), off, table.to(DEV), rows)
            assert not k.any() and not v.any()
            B.kv_cache_write(_cache(cache), q[:, :2], q[:, 2:4], off, lens, table.to(DEV))
        # 2 pages of the sequences' 19 and 5
        table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32)
        ref = R.attention64(q, t, off, lens, table, 0.1)
        lse = torch.empty((rows, 8), device=DEV)
        out = B.attention_paged(q, _cache(t), off, lens, table.to(DEV), max(new), scale=0.1, lse=lse)
        tol, tol_lse = R.attention_bounds(*ref, dim)
        assert ((out.double() - ref[0]).abs() <= tol).all() and ((lse.double() - ref[1]).abs() <= tol_lse).all()
    assert B.device_status() == B.OK


def test_a_longer_sequence_than_max_q_len(cuda_lib):
    """Its rows past max_q_len are left as they are; the others are right."""
    for cap, new in ((2, [5, 1]), (20, [150, 20])):
        t = R.make_cache(40, 2, 16, 128, 3, DEV)
        kv = [300, 64]
        off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
        table = R.make_table(kv, 16, 40, 19, 4)
        q = _randn((sum(new), 8, 128), 5)
        ref = R.attention64(q, t, off, lens, table, 0.1)
        out = torch.full_like(q, 6.0)
        B.attention_paged(q, _cache(t), off, lens, table.to(DEV), cap, scale=0.1, out=out)
        tol, _ = R.attention_bounds(*ref, 128)
        done = torch.zeros(sum(new), dtype=torch.bool, device=DEV)
        done[:cap] = True
        done[new[0]:] = True
        assert ((out.double() - ref[0]).abs() <= tol)[done].all() and (out[~done] == 6.0).all()


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [4, 2, 3, 4], [40, 41, 42, 43]])
def test_rows_that_see_nothing(cuda_lib, new):
    """Empty sequences, more new rows than tokens, absent pages: zeros and a log-sum of -inf."""
    for dim in (64, 128):
        _attend(2, 2, dim, 16, new, [0, 3, 100, 64], seed=40, absent=[(2, j) for j in range(7)], garbage=True)
        _attend(2, 2, dim, 16, new, [17, -5, 100, 200], seed=41, absent=[(2, 0), (2, 3), (3, 12)], window=20, garbage=True)


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [300, 90, 1000]), ([2, 1, 2], [5000, 0, 4000]), ([100, 30, 77], [400, 20, 1000]),
                                    ([900, 5, 1200], [900, 5, 1200])])
def test_not_a_number(cuda_lib, new, kv):
    """A NaN in a query or a decode scale shows in its row and head and nowhere else; rows without keys stay zeros."""
    for dim in (64, 128):
        t = R.make_cache(700, 2, 16, dim, 70, DEV)
        off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
        table = R.make_table(kv, 16, 700, max(-(-n // 16) for n in kv), 71).to(DEV)
        rows = sum(new)
        q = _randn((rows, 8, dim), 72)
        def run(q, t):
            lse = torch.full((rows, 8), 5.0, device=DEV)
            return B.attention_paged(q, _cache(t), off, lens, table, max(new), lse=lse), lse
        ref = R.attention64(q, t, off, lens, table, dim ** -0.5)
        tol, tol_lse = R.attention_bounds(*ref, dim)
        some = ~torch.isneginf(ref[1])
        bad = torch.zeros((rows, 8), dtype=torch.bool, device=DEV)
        bad[0, 3] = bad[rows - 1, 0] = bad[new[0], 5] = True
        qn = q.clone()
        qn[0, 3, 7] = qn[rows - 1, 0, 0] = qn[new[0], 5, dim - 1] = math.nan
        for name in (None, "g_k", "g_v"):
            if name is not None:
                bad = torch.zeros((rows, 8), dtype=torch.bool, device=DEV)
                bad[:, 4:] = True
                g = t[name].clone()
                g[1] = math.nan
            out, lse = run(qn, t) if name is None else run(q, {**t, name: g})
            hit = bad & some
            assert out[hit].isnan().all() and (name == "g_v" or lse[hit].isnan().all())
            assert ((out.double() - ref[0]).abs() <= tol)[~hit].all() and not out[~some].any()
            if name != "g_v":
                assert ((lse.double() - ref[1]).abs() <= tol_lse)[~hit & some].all()
            assert torch.equal(torch.isneginf(lse), ~some)
    assert B.device_status() == B.OK


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[1, 1], [200, 150]])
def test_large_scores(cuda_lib, dim, new):
    """Scores of hundreds: one key takes nearly all; growing maxima along the sequence."""
    _attend(2, 4, dim, 16, new, [500, 1500], seed=50, spread=20.0)
    _attend(2, 4, dim, 16, new, [500, 1500], seed=51, scale=-0.3)
    _attend(2, 4, dim, 16, new, [500, 1500], seed=52, scale=0.0)


@pytest.mark.parametrize("new", [[1, 1], [200, 150]])
def test_query_magnitudes(cuda_lib, new):
    """Queries far outside the range of 16-bit floats, zero rows, one element far above the others."""
    for std in (2.0 ** -40, 2.0 ** 30):
        q = _randn((sum(new), 8, 128), 60, std)
        q[0] = 0.0
        q[1, :, 5] *= 1000.0
        _attend(2, 4, 128, 16, new, [500, 700], seed=60, scale=0.09 / std, q=q)


@pytest.mark.parametrize("heads,group,dim,page,new,kv,window", [
    (4, 4, 128, 16, [1] * 64, [4096 - 61 * b for b in range(64)], 0),
    (8, 4, 128, 64, [1] * 3, [30000, 70, 12345], 0),
    (1, 8, 64, 16, [1], [65536], 0),
    (1, 1, 128, 16, [1] * 300, [1 + b for b in range(300)], 0),
    (2, 4, 128, 32, [700, 1000], [1900, 1000], 0),
    (8, 4, 128, 32, [512], [3000], 0),
    (16, 1, 64, 16, [256, 1, 100, 17, 200, 30, 256, 9], [5000, 4000, 100, 2000, 777, 30, 1500, 1025], 1024)])
def test_larger(cuda_lib, heads, group, dim, page, new, kv, window):
    _attend(heads, group, dim, page, new, kv, window, seed=70, garbage=len(kv) < 10)


def test_a_cache_past_32_bits(cuda_lib):
    """Byte offsets above 2^32 in the codes: 9 GB of pages, of which the far ones are used."""
    heads, dim, page, n_pages = 8, 128, 128, 70000
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("not enough free memory")
    t = {n: torch.zeros((n_pages, heads, page, d), dtype=torch.uint8, device=DEV)
         for n, d in (("k_codes", 64), ("v_codes", 64), ("k_scales", 8), ("v_scales", 8))}
    t["g_k"] = t["g_v"] = torch.full((heads,), 1 / 600, device=DEV)
    assert t["k_codes"].numel() > 1 << 32
    cache = _cache(t)
    far = [n_pages - 1, n_pages - 7, 3]
    kv, new = [300, 1], [300, 1]
    table = torch.tensor([far, [n_pages - 2, -1, -1]], dtype=torch.int32)
    off, lens = R.offsets(new), torch.tensor(kv, dtype=torch.int32)
    k, v, q = _randn((301, heads, dim), 1), _randn((301, heads, dim), 2), _randn((301, heads * 2, dim), 3)
    B.kv_cache_write(cache, k, v, off.to(DEV), lens.to(DEV), table.to(DEV))
    small = {n: (x[far + [n_pages - 2]].contiguous() if x.dim() == 4 else x) for n, x in t.items()}
    near = torch.tensor([[0, 1, 2], [3, -1, -1]], dtype=torch.int32)
    got = B.kv_cache_read(cache, off.to(DEV), table.to(DEV), 301)
    want = B.kv_cache_read(_cache(small), off.to(DEV), near.to(DEV), 301)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].any()
    ref = R.attention64(q, small, off.to(DEV), lens.to(DEV), near, 0.1)
    for rows, o, l in ((301, off, lens), (2, R.offsets([1, 1]), lens)):       # a chunk, and single tokens
        pick = torch.arange(301) if rows == 301 else torch.tensor([299, 300])
        out = B.attention_paged(q[pick.to(DEV)].contiguous(), cache, o.to(DEV), l.to(DEV), table.to(DEV),
                                300 if rows == 301 else 1, scale=0.1)
        tol, _ = R.attention_bounds(*(x[pick.to(DEV)] for x in ref), dim)
        assert ((out.double() - ref[0][pick.to(DEV)]).abs() <= tol).all()


@pytest.mark.parametrize("new,kv", [([1, 1, 1], [400, 90, 1000]), ([100, 30, 77], [400, 90, 1000])])
def test_strides_streams_and_graphs(cuda_lib, new, kv):
    """q as a slice of wider rows; another stream; two graphs captured from the
    same call, replayed at the same time on two streams; the same bits every time."""
    heads, group, dim, page = 2, 4, 128, 16
    n_pages = sum(-(-n // page) for n in kv) + 1
    t = R.make_cache(n_pages, heads, page, dim, 80, DEV)
    cache = _cache(t)
    table, off, lens = R.make_table(kv, page, n_pages, 64, 81).to(DEV), R.offsets(new).to(DEV), \
        torch.tensor(kv, dtype=torch.int32, device=DEV)
    wide = _randn((sum(new), heads * group * dim + 72), 82)
    q = wide[:, 8:8 + heads * group * dim].view(sum(new), heads * group, dim)
    call = lambda x=q: B.attention_paged(x, cache, off, lens, table, max(new))
    want = call(q.contiguous())
    assert torch.equal(call(), want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s1):
        other = call()
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    graphs, outs = [], []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call())
        graphs.append(g)
    for _ in range(20):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    assert B.device_status() == B.OK


def test_as_used_together(cuda_lib):
    """Rotate, write, attend, piece by piece and then token by token, against
    one call over the whole prompt and against 64 bits."""
    heads, group, dim, page = 2, 4, 128, 16
    lens = [150, 61]
    total = sum(lens)
    q, k, v = _randn((total, heads * group, dim), 90), _randn((total, heads, dim), 91), _randn((total, heads, dim), 92)
    freq = A.rope_frequencies(128, device=DEV)
    table = R.make_table(lens, page, 16, 12, 93).to(DEV)
    first = R.offsets(lens).tolist()

    def serve(pieces):
        cache = A.KVCache.empty(16, page, heads, dim, 6.0, 5.0, DEV)
        out = torch.zeros_like(q)
        done = [0, 0]
        for new in pieces:
            rows = torch.cat([torch.arange(first[b] + done[b], first[b] + done[b] + n) for b, n in enumerate(new)]).to(DEV)
            pos = torch.cat([torch.arange(done[b], done[b] + n) for b, n in enumerate(new)]).to(DEV)
            done = [d + n for d, n in zip(done, new)]
            qr, kr = B.rope(q[rows], k[rows], pos, freq)
            off, kv = R.offsets(new).to(DEV), torch.tensor(done, dtype=torch.int32, device=DEV)
            B.kv_cache_write(cache, kr, v[rows], off, kv, table)
            out[rows] = B.attention_paged(qr, cache, off, kv, table, max(new))
        return out, cache

    whole, cache = serve([lens])
    parts, cache2 = serve([[64, 30], [40, 1], [40, 25]] + [[1, 1]] * 5 + [[1, 0]])
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(cache, n), getattr(cache2, n))
    t = {n: getattr(cache, n) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "g_k", "g_v")}
    qr = B.rope(q, None, torch.cat([torch.arange(n) for n in lens]).to(DEV), freq)[0]
    ref = R.attention64(qr, t, R.offsets(lens).to(DEV), torch.tensor(lens, device=DEV), table, dim ** -0.5)
    tol, _ = R.attention_bounds(*ref, dim)
    for o in (whole, parts):
        assert ((o.double() - ref[0]).abs() <= tol).all()
    # what the trainer reads back is what was attended
    kb, vb = B.kv_cache_read(cache, R.offsets(lens).to(DEV), table, total, out_dtype=B.OUT_F32)
    kv64 = R.values64(t, "k")
    b0 = table[0, :10].long().cpu()
    want = torch.cat([kv64[p].transpose(0, 1) for p in b0])[:150]
    assert torch.equal(kb[:150], want.float())
