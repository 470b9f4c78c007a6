"""The layer stack with attention over the NVFP4 KV cache on both sides."""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import kvcache as K
from oracle import nvfp4 as Q
from tests import kvcache_ref as R
from train_alignment_b200 import attention as A
from train_alignment_b200 import stack as ST
from train_alignment_b200 import workloads as W

pytestmark = pytest.mark.gpu

CFG = W.MoEConfig("stack3_t300_h256_e8k2_f256", T=300, H=256, E=8, k=2, F=256, n_chan=16, n_chan_f=16, n_outlier=3,
                  outlier_scale=16.0, layers=3)
ATTN = W.AttnConfig(heads_q=4, heads_k=2, dim=64, rot=32, page=16, n_seqs=3)


def _parts(cache):
    return {n: getattr(cache, n) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "g_k", "g_v")}


def _check_attention(a, x, cache, got):
    """A layer's attention from its own rotated queries and cache, in 64 bits."""
    q, _, _ = a.project(x)
    ref = R.attention64(q, _parts(cache), a.off, a.kv_len, a.table, a.cfg.dim ** -0.5, a.cfg.window)
    tol, _ = R.attention_bounds(*ref, a.cfg.dim)
    assert ((got.double() - ref[0]).abs() <= tol).all()


@pytest.mark.parametrize("attn", [ATTN, dataclasses.replace(ATTN, interleaved=True, window=40, dim=128, rot=128)])
def test_stack_with_attention(cuda_lib, attn):
    st = ST.LayerStack(CFG, seed=1, device="cuda", recorded=1, attn=attn)
    gap, cm, sm = st.alignment_pass(drift=1e-3)
    assert cuda_lib.device_status() == cuda_lib.OK
    assert torch.isfinite(gap).all() and gap.shape == (CFG.T,)
    for l, a in enumerate(st.attn):
        x = st.x_roll[l]
        q, k, v = a.project(x)
        # the rotation, and the cache, against the oracle
        c = a.cfg
        qkv = (x @ a.w_qkv.t()).view(CFG.T, -1, c.dim)
        ref = K.rope(qkv[:, :c.heads_q].double().cpu().numpy(), a.pos.cpu().numpy(), a.freq.cpu().numpy(), c.interleaved)
        mag = np.abs(qkv[:, :c.heads_q].double().cpu().numpy()).max()
        assert (np.abs(q.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * mag).all()
        kr, vr = cuda_lib.kv_cache_read(a.cache, a.off, a.table, CFG.T, out_dtype=cuda_lib.OUT_F32)
        for t, r, g in ((k, kr, a.cache.g_k), (v, vr, a.cache.g_v)):
            for h in range(c.heads_k):
                codes, scales = Q.quantize_with_scale(t[:, h].double().cpu().numpy(), float(g[h]))
                want = np.float32(Q.dequant(codes, scales, float(g[h])))
                np.testing.assert_array_equal(r[:, h].cpu().numpy(), want)
        o = cuda_lib.attention_paged(q, a.cache, a.off, a.kv_len, a.table, a.longest, window=c.window)
        _check_attention(a, x, a.cache, o)
        # x_mid is the residual sum of that attention's projection
        mid = cuda_lib.residual_add(x, o.view(CFG.T, -1) @ a.w_o.t())
        assert torch.equal(mid, st.x_mid[l])
        # the trainer attended over the rollout's cache where it is recorded, over its own elsewhere
        xt = st.x_train[l]
        cache = a.cache if st.is_recorded(l) else a.t_cache
        qt, kt, vt = a.project(xt)
        ot = cuda_lib.attention_paged(qt, cache, a.off, a.kv_len, a.table, a.longest, window=c.window)
        _check_attention(a, xt, cache, ot)
        assert torch.equal(cuda_lib.residual_add(xt, ot.view(CFG.T, -1) @ a.w_o.t()), st.x_mid_train[l])
    # the recorded MoE layer replays its own input (the attention's output) without a mismatch
    layer = st.layers[2]
    layer.reset_counts()
    layer.trainer_replay(st.x_mid[2], layer_id=2)
    assert int(layer.status.item()) == 0 and layer.counts.tolist() == [0, 0]
    gaps = st.kv_gaps()
    assert list(gaps) == [2] and all(0.0 < g < 0.5 for g in gaps[2])


def test_trainer_without_drift_attends_alike(cuda_lib):
    """With the rollout's own input the first layer's trainer writes the same
    cache and gets the same attention, bit for bit."""
    st = ST.LayerStack(CFG, seed=2, device="cuda", recorded=0, attn=ATTN)
    a = st.attn[0]
    assert torch.equal(a.rollout(st.x0), a.trainer(st.x0, replay=False))
    assert torch.equal(a.trainer(st.x0, replay=True), a.trainer(st.x0, replay=False))
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(a.cache, n), getattr(a.t_cache, n))


def test_w4a4_ablation_with_attention(cuda_lib):
    st = ST.LayerStack(CFG, seed=3, device="cuda", recorded=2, attn=ATTN)
    gap, cm, sm = st.alignment_pass(drift=1e-3, w4a4=True)
    assert torch.isfinite(gap).all() and (cm, sm) == (0, 0)
    assert cuda_lib.device_status() == cuda_lib.OK


def test_the_named_configuration(cuda_lib):
    """The 2048-hidden stack's attention shape on two layers."""
    cfg = dataclasses.replace(W.STACK8_T4096, layers=2)
    st = ST.LayerStack(cfg, seed=0, device="cuda", recorded=1, attn=W.ATTN_H2048)
    gap, cm, sm = st.alignment_pass()
    assert torch.isfinite(gap).all() and cuda_lib.device_status() == cuda_lib.OK
    a = st.attn[1]
    q, _, _ = a.project(st.x_roll[1])
    o = cuda_lib.attention_paged(q, a.cache, a.off, a.kv_len, a.table, a.longest)
    _check_attention(a, st.x_roll[1], a.cache, o)
    assert isinstance(a, A.CachedAttention)
