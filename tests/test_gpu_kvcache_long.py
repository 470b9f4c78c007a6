"""Attention over contexts of 2^18 to 2^31 tokens.  Every entry of the block
table names the same page, so the cache is small and a softmax over the
positions is one over the page's places, each as often as it is seen."""
import math

import pytest
import torch

from tests import kvcache_ref as R
from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE = 65536


def _long(heads, group, dim, kv, new, window=0, seed=1):
    """out, lse of one call and the error bounds of its rows: (out, lse, ref, ref_lse, vabs)."""
    t = R.make_cache(1, heads, PAGE, dim, seed, DEV)
    t["v_codes"] &= 0x77                                 # values of one sign, so that nothing averages out
    cache = A.KVCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], t["g_k"], t["g_v"])
    table = torch.zeros((len(kv), -(-max(kv) // PAGE)), dtype=torch.int32, device=DEV)
    off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
    q = (torch.randn((sum(new), heads * group, dim), generator=torch.Generator().manual_seed(seed + 1)) * 0.3).to(torch.bfloat16)
    q = q.to(DEV)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = B.attention_paged(q, cache, off, lens, table, max(new), window=window, lse=lse)
    assert B.device_status() == B.OK
    k, v = R.values64(t, "k")[0], R.values64(t, "v")[0]
    slot = torch.arange(PAGE, device=DEV)
    upto = lambda p: torch.div(p - slot + PAGE, PAGE, rounding_mode="floor").clamp_min(0)     # positions <= p at each place
    rows = sorted({0, new[0] // 2, new[0] - 1, sum(new) // 2, sum(new) - 1})
    ref, ref_lse, first = [], [], off.tolist()
    for r in rows:
        b = max(i for i in range(len(kv)) if first[i] <= r)
        pos = kv[b] - new[b] + r - first[b]
        n = upto(pos) - (upto(pos - window) if window else 0)
        s = torch.einsum("hd,lhd->hl", q[r].double(), k.transpose(0, 1).repeat_interleave(group, 1)) * dim ** -0.5
        s = s + torch.log(n.double())
        ref_lse.append(torch.logsumexp(s, -1))
        ref.append(torch.einsum("hl,hld->hd", torch.softmax(s, -1), v.repeat_interleave(group, 0)))
    return out[rows].double(), lse[rows].double(), torch.stack(ref), torch.stack(ref_lse)


def _check(got, lse, ref, ref_lse):
    # values are positive, so the weighted |v| is the result itself.  Weights
    # rounded to 16 bits and their exponentials as in attention_bounds; a matrix
    # instruction adds the products of 16 keys to a sum in 32 bits, truncating
    # both: off by at most 2 * 2^-23 of it.  Of at most 4096 additions to a sum
    # that grows evenly that is 2^-11 of the last, and the same again for what
    # is added after (in 32 bits, rounded) and the scores (dim 2^-23 of theirs).
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12) * ref.abs()
    assert ((got - ref).abs() <= tol).all(), ((got - ref).abs() / ref.abs()).max()
    assert ((lse - ref_lse).abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,kv,new", [
    (8, 4, [1 << 20], [2560]), (8, 4, [1 << 18, (1 << 18) - 5], [1100, 1400]), (1, 4, [(1 << 23) - 3], [64]),
    (8, 4, [(1 << 22) + 70000], [320]), (4, 4, [1 << 21], [700])])
def test_long_sums_of_chunks(cuda_lib, dim, heads, group, kv, new):
    """Sums of so many keys in one block (and in parts) that additions which truncate would show."""
    _check(*_long(heads, group, dim, kv, new))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,kv,new", [
    (8, 1, [1 << 22] * 64, [1] * 64), (8, 4, [(1 << 22) - 77] * 64, [4] * 64), (1, 1, [1 << 30], [1]),
    (8, 4, [(1 << 22) + 5, 300] * 40, [1, 2] * 40)])
def test_long_sums_of_few_rows(cuda_lib, dim, heads, group, kv, new):
    """The same of the kernel for few rows, where a CTA's run is long."""
    _check(*_long(heads, group, dim, kv, new))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,length,new", [(8, 4, 1 << 20, [2560]), (1, 4, 1 << 22, [64]), (8, 1, 1 << 22, [1] * 64),
                                                    (8, 4, (1 << 22) - 99, [4] * 64)])
def test_long_sums_whose_maximum_grows(cuda_lib, dim, heads, group, length, new):
    """Sums kept in memory at one maximum and continued at another: the last
    page's scores are 9.5 powers of two above those of all pages before, whose
    keys weigh enough together to be seen."""
    t = R.make_cache(2, heads, PAGE, dim, 3, DEV)
    t["k_scales"].fill_(0x38)
    t["g_k"] = torch.ones(heads, device=DEV)
    t["k_codes"][0], t["k_codes"][1] = 0x22, 0x33        # 1 and 1.5 in every element
    t["v_codes"] &= 0x77
    cache = A.KVCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], t["g_k"], t["g_v"])
    table = torch.zeros((len(new), -(-length // PAGE)), dtype=torch.int32, device=DEV)
    table[:, -1] = 1
    off, lens = R.offsets(new).to(DEV), torch.full((len(new),), length, dtype=torch.int32, device=DEV)
    rows, scale = sum(new), 9.5 * math.log(2.0) * 2 / dim
    q = torch.ones((rows, heads * group, dim), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((rows, heads * group), device=DEV)
    out = B.attention_paged(q, cache, off, lens, table, max(new), scale=scale, lse=lse)
    assert B.device_status() == B.OK
    v = R.values64(t, "v")                               # [2, heads, places, dim]
    total, full = v.sum(2), (table.shape[1] - 1)
    for r in (0, rows // 2, rows - 1):
        b = max(i for i in range(len(new)) if int(off[i]) <= r)
        pos = length - new[b] + r - int(off[b])
        last = pos - full * PAGE + 1                     # keys of the last page that it sees
        w = 2.0 ** 9.5
        den = full * PAGE + w * last
        ref = (full * total[0] + w * v[1, :, :last].sum(1)) / den
        _check(out[r].double(), lse[r].double(), ref.repeat_interleave(group, 0),
               torch.full((heads * group,), scale * dim + math.log(den), dtype=torch.float64, device=DEV))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("window", [(1 << 30) - 12345, (1 << 30) + (1 << 28) + 77])
def test_windows_around_2_to_the_30(cuda_lib, dim, new, window):
    """Windows past 2^30 are as long as they say."""
    kv = (1 << 30) + (1 << 29) - 54321
    # the places of a part of a page are seen once more than the others: too little to be seen here, so
    # the log-sum tells the windows apart: 2^-14 of 2^30 positions are 2^16
    _check(*_long(1, 1, dim, [kv], [new], window=window))
