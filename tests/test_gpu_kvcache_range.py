"""Attention over the NVFP4 KV cache at the ends of its number range."""
import math

import pytest
import torch

from tests import kvcache_ref as R
from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (key heads, query heads of each, new, cached): a context taken whole, contexts
# cut into runs and joined, groups of rows, chunks, chunks whose keys are split
SHAPES = [(2, 4, [1, 1], [700, 40]), (2, 4, [1, 1], [5000, 300]), (1, 1, [1], [20000]), (1, 16, [3, 2], [1100, 2]),
          (8, 4, [3, 2], [1500, 1500]), (2, 4, [100, 20], [300, 20]), (1, 1, [100], [6000]), (1, 4, [300, 100], [2000, 5000])]


def _cache(t):
    return A.KVCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], t["g_k"], t["g_v"])


def _plain_keys(heads, new, kv, dim, page=16, seed=1, far=()):
    """A cache whose keys are all 2 in every element, but 1 at the positions
    `far` of each sequence (scale bytes 1.0, decode scales 1); random values."""
    n_pages = sum(-(-n // page) for n in kv) + 2
    t = R.make_cache(n_pages, heads, page, dim, seed, DEV)
    table = R.make_table(kv, page, n_pages, max(-(-n // page) for n in kv), seed + 1)
    t["k_codes"].fill_(0x44)
    t["k_scales"].fill_(0x38)
    t["g_k"] = torch.ones(heads, device=DEV)
    for b, n in enumerate(kv):
        for j in far:
            if j < n:
                t["k_codes"][int(table[b, j // page]), :, j % page] = 0x22
    return t, table


def _call(q, t, new, kv, table, scale, window=0):
    off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    B.attention_paged(q, _cache(t), off, lens, table.to(DEV), max(new), scale=scale, window=window, out=out, lse=lse)
    assert B.device_status() == B.OK
    return out, lse, R.attention64(q, t, off, lens, table, scale, window)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new,kv", SHAPES)
def test_scores_far_below_zero(cuda_lib, dim, heads, group, new, kv):
    """All scores of a row about -1e35: the rows attend as at any other
    magnitude.  Scores are a power of two times one factor, so equal ones are
    equal in 32 bits too: a row takes the key of half the score once it sees
    it, and the mean of all before."""
    for far in ((), (17,), (299,), (4000, 31)):
        t, table = _plain_keys(heads, new, kv, dim, seed=3, far=far)
        q = torch.ones((sum(new), heads * group, dim), dtype=torch.bfloat16, device=DEV)
        out, lse, ref = _call(q, t, new, kv, table, -1e33)
        tol = 2.0 ** -8 * ref[0].abs() + (2.0 ** -11 + 2.0 ** -15) * ref[2] * (1 + 2.0 ** -7) + 1e-30
        assert ref[1].max() < -5e34 and ((out.double() - ref[0]).abs() <= tol).all()
        # the factor is a product of five numbers, each rounded to 32 bits, and the change of base another
        assert ((lse.double() - ref[1]).abs() <= 2.0 ** -20 * ref[1].abs()).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new,kv", SHAPES)
def test_infinities(cuda_lib, dim, heads, group, new, kv):
    """A query with an infinite element, and a head with an infinite decode
    scale, have no softmax: NaNs, in that row and head and nowhere else.  With
    keys of one sign every score of such a row is -inf, or every one +inf."""
    t, table = _plain_keys(heads, new, kv, dim, seed=5)
    rows, hq = sum(new), heads * group
    q = torch.ones((rows, hq, dim), dtype=torch.bfloat16, device=DEV)
    scale = dim ** -0.5
    for at, x in ((5, -math.inf), (dim - 1, math.inf)):
        for r, h in ((0, hq - 1), (rows - 1, 0)):
            qx = q.clone()
            qx[r, h, at] = x
            hit = torch.zeros((rows, hq), dtype=torch.bool, device=DEV)
            hit[r, h] = True
            out, lse, _ = _call(qx, t, new, kv, table, scale)
            ref = R.attention64(q, t, R.offsets(new), torch.tensor(kv), table, scale)
            tol, tol_lse = R.attention_bounds(*ref, dim)
            assert out[hit].isnan().all() and lse[hit].isnan().all()
            assert ((out.double() - ref[0]).abs() <= tol)[~hit].all()
            assert ((lse.double() - ref[1]).abs() <= tol_lse)[~hit].all()
    for name in ("g_k", "g_v"):
        for x in (-math.inf, math.inf):
            g = t[name].clone()
            g[heads - 1] = x
            out, lse, _ = _call(q, {**t, name: g}, new, kv, table, scale)
            assert out[:, -group:].isnan().all() and (name == "g_v" or lse[:, -group:].isnan().all())
            assert not out[:, :-group].isnan().any() and not lse[:, :-group].isnan().any()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,new,kv", SHAPES)
def test_scores_past_32_bits(cuda_lib, dim, heads, group, new, kv):
    """Scores that are all -inf in 32 bits: NaNs, not the zeros of a row that sees nothing."""
    t, table = _plain_keys(heads, new, kv, dim, seed=6)
    q = torch.ones((sum(new), heads * group, dim), dtype=torch.bfloat16, device=DEV)
    out, lse, _ = _call(q, t, new, kv, table, -1e37)
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv", [([3, 4, 1], [2, 400, 500]), ([3, 4, 1], [2, 4000, 2000]), ([200, 90, 130], [150, 400, 700]),
                                    ([100, 70, 90], [60, 5000, 90])])
def test_infinities_in_rows_that_see_nothing(cuda_lib, dim, new, kv):
    """Zeros and a log-sum of -inf where no position is visible: before position
    0, or with a window whose pages are absent although others are there."""
    heads, group, window = 2, 4, 20
    t, table = _plain_keys(heads, new, kv, dim, seed=7)
    table[1, 2:] = -1                                    # positions from 32 on: windows from 51 on see nothing
    q = torch.full((sum(new), heads * group, dim), -math.inf, dtype=torch.bfloat16, device=DEV)
    out, lse, _ = _call(q, t, new, kv, table, 0.1, window)
    b = torch.repeat_interleave(torch.arange(3), torch.tensor(new))
    i = torch.cat([torch.arange(n) for n in new])
    pos = torch.tensor(kv)[b] - torch.tensor(new)[b] + i
    sees = ((pos >= 0) & ((b != 1) | (pos - window + 1 < 32))).to(DEV)
    assert 0 < int(sees.sum()) < len(pos)
    assert out[sees].isnan().all() and lse[sees].isnan().all()
    assert not out[~sees].any() and torch.isneginf(lse[~sees]).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 18, 2.0 ** 24])
@pytest.mark.parametrize("heads,group,new,kv", SHAPES[:7])
def test_a_query_of_wide_spread(cuda_lib, dim, ratio, heads, group, new, kv):
    """One element `ratio` times the others, where every key is zero: the scores
    are those of the others, to 32 bits."""
    n_pages = sum(-(-n // 16) for n in kv) + 2
    t = R.make_cache(n_pages, heads, 16, dim, 8, DEV)
    t["k_codes"][..., 3] &= 0x0F                         # element 7
    table = R.make_table(kv, 16, n_pages, max(-(-n // 16) for n in kv), 9)
    g = torch.Generator().manual_seed(10)
    q = torch.randn((sum(new), heads * group, dim), generator=g).to(torch.bfloat16).to(DEV)
    q[..., 7] = ratio
    out, lse, ref = _call(q, t, new, kv, table, dim ** -0.5)
    tol, tol_lse = R.attention_bounds(*ref, dim)
    assert ((out.double() - ref[0]).abs() <= tol).all() and ((lse.double() - ref[1]).abs() <= tol_lse).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_read_without_a_page_beside_a_scale_that_is_not_a_number(cuda_lib, dim):
    """Zeros where there is no page, whatever the head's decode scale."""
    t = R.make_cache(4, 2, 16, dim, 11, DEV)
    t["g_k"][1] = math.nan
    t["g_v"][0] = math.inf
    off = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    table = torch.tensor([[2, -1, 1]], dtype=torch.int32, device=DEV)
    for dt in (B.OUT_F32, B.OUT_BF16):
        k, v = B.kv_cache_read(_cache(t), off, table, 40, out_dtype=dt)
        assert not k[16:32].any() and not v[16:32].any()
        assert k[:16, 1].isnan().all() and k[32:, 0].any() and not k[:, 0].isnan().any() and not v[:, 1].isnan().any()


def _range(q, t, new, kv, table, scale):
    """Per row and head: the least and greatest of each element among the values
    of the keys whose 64-bit scores are within 2 d of the largest, d = dim 2^-23
    + 2^-22 of the largest sum of |terms| (what scores in 32 bits can be off
    by), and 40 more (the others weigh less than 2^-57 each); the largest score;
    d."""
    k, v = R.values64(t, "k"), R.values64(t, "v")
    (rows, hq, dim), heads, page = q.shape, k.shape[1], k.shape[2]
    lo, hi = torch.empty((2, rows, hq, dim), dtype=torch.float64, device=DEV)
    top, far = torch.empty((2, rows, hq), dtype=torch.float64, device=DEV)
    r0 = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        j = torch.arange(length)
        at, place = table[b, j // page].long().to(DEV), (j % page).to(DEV)
        see = j.to(DEV)[None] <= torch.arange(length - n, length, device=DEV)[:, None]
        for h in range(hq):
            kk, vv = k[at, h * heads // hq, place], v[at, h * heads // hq, place]
            x = q[r0:r0 + n, h].double()
            s = (x @ kk.T * scale).masked_fill(~see, -math.inf)
            m = s.amax(1, keepdim=True)
            d = (x.abs() @ kk.abs().T * abs(scale)).masked_fill(~see, 0.0).amax(1, keepdim=True) * (dim * 2.0 ** -23 + 2.0 ** -22)
            for i in range(n):
                near = vv[(s[i] >= m[i] - 2 * d[i] - 40)]
                lo[r0 + i, h], hi[r0 + i, h] = near.amin(0), near.amax(0)
            top[r0:r0 + n, h], far[r0:r0 + n, h] = m[:, 0], d[:, 0]
        r0 += n
    return lo, hi, top, far


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8, 1e10, 1e20, 1e30])
@pytest.mark.parametrize("heads,group,new,kv", SHAPES)
def test_huge_scores(cuda_lib, dim, size, heads, group, new, kv):
    """Finite scores of any size and both signs: a row is a mean of the values of
    the keys that scores in 32 bits cannot tell from the first, mostly one."""
    n_pages = sum(-(-n // 16) for n in kv) + 2
    t = R.make_cache(n_pages, heads, 16, dim, 12, DEV)
    table = R.make_table(kv, 16, n_pages, max(-(-n // 16) for n in kv), 13)
    g = torch.Generator().manual_seed(14)
    q = torch.randn((sum(new), heads * group, dim), generator=g).to(torch.bfloat16).to(DEV)
    for scale in (size, -size):
        off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
        lse = torch.empty(q.shape[:2], device=DEV)
        out = B.attention_paged(q, _cache(t), off, lens, table.to(DEV), max(new), scale=scale, lse=lse).double()
        assert B.device_status() == B.OK and not out.isnan().any() and not lse.isnan().any()
        lo, hi, top, d = _range(q, t, new, kv, table, scale)
        # a weight and a sum rounded as in attention_bounds, of values at most the range's largest; rounding to BF16
        tol = (2.0 ** -8 + 2.0 ** -10) * torch.maximum(lo.abs(), hi.abs()) + 2.0 ** -30
        assert ((out >= lo - tol) & (out <= hi + tol)).all()
        assert (lo == hi).all(-1).float().mean() > 0.9
        assert ((lse.double() - top).abs() <= d + math.log(max(kv)) + 2.0 ** -20 * top.abs()).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv,rows", [([3, 6], [40, 50], 5), ([3, 6], [2000, 1500], 5), ([90, 120], [300, 400], 150),
                                         ([100], [6000], 70), ([5], [3], 4)])
def test_fewer_rows_than_the_offsets_name(cuda_lib, dim, new, kv, rows):
    """Rows have the positions that the offsets give them, also where the call
    ends before the last sequence does."""
    t = R.make_cache(800, 2, 16, dim, 15, DEV)
    table = R.make_table(kv, 16, 800, max(-(-n // 16) for n in kv), 16)
    off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
    q = torch.randn((sum(new), 8, dim), generator=torch.Generator().manual_seed(17)).to(torch.bfloat16).to(DEV)
    ref = R.attention64(q, t, off, lens, table, 0.1)
    tol, tol_lse = (x[:rows] for x in R.attention_bounds(*ref, dim))
    lse = torch.empty((rows, 8), device=DEV)
    out = B.attention_paged(q[:rows], _cache(t), off, lens, table.to(DEV), max(new), scale=0.1, lse=lse)
    empty = torch.isneginf(ref[1][:rows])
    assert ((out.double() - ref[0][:rows]).abs() <= tol).all() and torch.equal(torch.isneginf(lse), empty)
    assert ((lse.double() - ref[1][:rows])[~empty].abs() <= tol_lse[~empty]).all()
