"""Attention over the NVFP4 KV cache at the ends of its number range."""
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
