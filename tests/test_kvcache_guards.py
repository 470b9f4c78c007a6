"""What the KV cache's Python side refuses or rebuilds, on the host."""
import copy
import io
import struct

import pytest
import torch

from train_alignment_b200 import attention as A
from train_alignment_b200 import binding as B

TENSORS = ("k_codes", "k_scales", "v_codes", "v_scales", "g_k", "g_v")


def _addresses(cache):
    return struct.unpack("@qiiii6Q", cache.desc)[5:]


def _own(cache):
    return tuple(getattr(cache, n).data_ptr() for n in TENSORS)


@pytest.mark.parametrize("name", TENSORS + ("desc", "n_pages", "page_size", "n_heads", "head_dim", "other"))
def test_a_cache_keeps_its_tensors(name):
    """Calls go by the addresses taken when the cache was made: no attribute can
    be set to another tensor behind them."""
    c = A.KVCache.empty(3, 16, 2, 64, 6.0, 6.0, device="cpu")
    before = dict(c.__dict__)
    with pytest.raises(AttributeError):
        setattr(c, name, torch.zeros_like(c.k_codes))
    if name != "other":
        with pytest.raises(AttributeError):
            delattr(c, name)
    assert c.__dict__.keys() == before.keys() and all(c.__dict__[n] is x for n, x in before.items())
    assert _addresses(c) == _own(c)


def test_copies_describe_their_own_tensors():
    c = A.KVCache.empty(3, 16, 2, 64, 6.0, 6.0, device="cpu")
    c.k_codes.fill_(7)
    buf = io.BytesIO()
    torch.save(c, buf)
    buf.seek(0)
    same, deep, loaded = copy.copy(c), copy.deepcopy(c), torch.load(buf, weights_only=False)
    assert _own(same) == _own(c) and not set(_own(deep)) & set(_own(c)) and not set(_own(loaded)) & set(_own(c))
    for x in (same, deep, loaded):
        assert _addresses(x) == _own(x) and x.page_size == 16 and x.head_dim == 64
        for n in TENSORS:
            assert torch.equal(getattr(x, n), getattr(c, n))


def test_gradients_are_not_cut_in_silence():
    """Arguments that require a gradient are refused while autograd records, and
    pass on to the other checks (here: host tensors) where it does not."""
    c = A.KVCache.empty(3, 32, 2, 64, 6.0, 6.0, device="cpu")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    y = x.clone().requires_grad_()
    i = torch.zeros(2, dtype=torch.int32)
    pos, freq = torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    learned = freq.clone().requires_grad_()
    calls = [lambda: B.kv_cache_write(c, y, x, i, i[:1], i.view(1, 2)), lambda: B.kv_cache_write(c, x, y * 2, i, i[:1], i.view(1, 2)),
             lambda: B.attention_paged(y, c, i, i[:1], i.view(1, 2), 4), lambda: B.rope(y, None, pos, freq),
             lambda: B.rope(x, y, pos, freq), lambda: B.rope(x, None, pos, learned),
             lambda: B.rope_backward(x, y, pos, freq)]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
        with torch.inference_mode(), pytest.raises(ValueError, match="CUDA"):
            call()
    parts = [getattr(c, n) for n in TENSORS]
    for at in (4, 5):
        with pytest.raises(ValueError, match="detached"):
            A.KVCache(*[p.clone().requires_grad_() if j == at else p for j, p in enumerate(parts)])
