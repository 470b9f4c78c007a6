"""Chunks whose keys are split many ways, the cache's calls in a CUDA graph, and
the attention's bounded waits."""
import pytest
import torch

from tests import kvcache_ref as R
from tests.test_gpu_kvcache import DEV, _attend, _cache, _randn
from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B

pytestmark = pytest.mark.gpu


def _splits(heads, group, dim, page, rows, n_seqs, longest, max_q_len):
    """Ways that a chunk's keys are split, from the workspace that holds their parts."""
    c = A.KVCache.empty(1, page, heads, dim, 1.0, 1.0, DEV)
    width = -(-longest // page)
    need = B.attention_paged_workspace_bytes(c, rows, heads * group, n_seqs, width, max_q_len)
    part = rows * heads * group * (4 * dim + 8)
    assert need % part == 0
    return need // part


# at least so many parts on 148 SMs: more than a warp has lanes, the lanes' last
# batch partly filled, parts that a window leaves empty, a short sequence beside
# a long one, and parts cut back to what 256 MB hold
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,page,new,kv,extra,least", [
    (1, 1, 16, [100], [65536], 0, 100), (1, 1, 16, [100], [20000], 2, 33), (1, 1, 128, [100, 70], [65536, 300], 1, 40),
    (1, 8, 64, [256], [65536], 0, 10), (2, 4, 16, [60, 20], [9000, 9000], 0, 10), (1, 1, 64, [100], [65536], 20000, 20)])
@pytest.mark.parametrize("window", [0, 200, 7000])
def test_many_parts(cuda_lib, dim, heads, group, page, new, kv, extra, least, window):
    n = _splits(heads, group, dim, page, sum(new) + extra, len(kv), max(kv), max(new))
    assert n >= least and (extra < 1000 or n * (sum(new) + extra) * heads * group * (4 * dim + 8) <= 1 << 28)
    _attend(heads, group, dim, page, new, kv, window, seed=60, extra=extra)


@pytest.mark.parametrize("dim,inter", [(64, True), (128, False)])
def test_rotate_write_and_read_in_a_graph(cuda_lib, dim, inter):
    """Captured once and replayed on new inputs, on two streams in turn: the same bits as called."""
    heads, page, new, kv = 2, 16, [40, 1, 70], [100, 33, 70]
    rows, n_pages = sum(new), sum(-(-n // page) for n in kv) + 1
    off, lens = R.offsets(new).to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV)
    start = lens - (off[1:] - off[:-1])
    table = R.make_table(kv, page, n_pages, 7, 3).to(DEV)
    pos = torch.cat([torch.arange(k - n, k) for n, k in zip(new, kv)]).to(DEV)
    freq = A.rope_frequencies(dim // 2, device=DEV)
    q, k, v = (_randn((rows, h, dim), s) for h, s in ((4, 1), (heads, 2), (heads, 3)))
    cache = A.KVCache.empty(n_pages, page, heads, dim, 5.0, 5.0, DEV)

    def step(c):
        qr, kr = B.rope(q, k, pos, freq, interleaved=inter)
        B.kv_cache_write(c, kr, v, off, lens, table)
        return (qr, kr, *B.kv_cache_read(c, off, table, rows, start=start, out_dtype=B.OUT_F32),
                *B.rope_backward(qr, kr, pos, freq, interleaved=inter))

    step(cache)
    graph, s1, s2 = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s1):
        outs = step(cache)
    for i in range(4):
        for x, s in ((q, 10), (k, 20), (v, 30)):
            x.copy_(_randn(x.shape, s + i))
        other = A.KVCache.empty(n_pages, page, heads, dim, 5.0, 5.0, DEV)
        want = step(other)
        torch.cuda.synchronize()
        with torch.cuda.stream((s1, s2)[i % 2]):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(cache, n), getattr(other, n))
    assert B.device_status() == B.OK


def test_a_wait_that_runs_out_is_reported_once(cuda_lib):
    """Each of the two records of timeouts is read and cleared, and a call works after."""
    tests = (B.selftest_attention_wait, B.selftest_bounded_wait)
    for calls in (tests[:1], tests[1:], tests):
        assert B.device_status() == B.OK
        for f in calls:
            f(2_000_000)                               # 2 ms on a barrier that nothing completes
        assert B.device_status() == B.ERR_TIMEOUT and B.device_status() == B.OK
    _attend(2, 4, 64, 16, [100], [300], seed=61)
