"""Host-side checks of the serving operators, no GPU: refusals before any
launch, workspace plans, and pins of their oracles."""
import math

import numpy as np
import pytest
import torch

import fsq_latent_decode_b200 as F
from oracle import fsq_oracle as O


# ---------------------------------------------------------------- head norms + rotary positions
def _norm_rope(**kw):
    a = dict(q=1 << 20, ldq=4096, n_q=32, qg=None, qo=2 << 20, ldqo=4096, k=3 << 20, ldk=1024, n_k=8, kg=None,
             ko=4 << 20, ldko=1024, n=5, d=128, pos=None, pos0=0, eps=1e-6, base=1e6, stream=None)
    a.update(kw)
    return F.qk_norm_rope_raw(*a.values())


def test_norm_rope_refusals():
    bad, un, mis = F.FSQ_ERR_INVALID_ARG, F.FSQ_ERR_UNSUPPORTED, F.FSQ_ERR_MISALIGNED
    assert _norm_rope(n=0, q=None, qo=None) == F.FSQ_OK
    for kw in (dict(n=-1), dict(n_q=0), dict(n_k=-1), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None),
               dict(ldq=4088), dict(ldqo=4088), dict(ldk=1016), dict(ldko=1016), dict(eps=-1.0),
               dict(eps=math.nan), dict(eps=math.inf), dict(base=1.0), dict(base=math.nan), dict(base=math.inf)):
        assert _norm_rope(**kw) == bad, kw
    for kw in (dict(d=64), dict(n_q=65535), dict(n=1 << 31)):
        assert _norm_rope(**kw) == un, kw
    for kw in (dict(q=(1 << 20) + 8), dict(qo=(2 << 20) + 2), dict(k=(3 << 20) + 8), dict(ko=(4 << 20) + 8),
               dict(ldq=4100), dict(ldqo=4100), dict(ldk=1028), dict(ldko=1028), dict(qg=8), dict(kg=8),
               dict(pos=2)):
        assert _norm_rope(**kw) == mis, kw


def test_norm_rope_refuses_overlaps():
    bad = F.FSQ_ERR_INVALID_ARG
    q = 1 << 20
    assert _norm_rope(qo=q + 4096) == bad                            # half a row into the input
    assert _norm_rope(qo=q, ldqo=8192) == bad                         # the input with another stride
    assert _norm_rope(ko=q + 4096 * 2 * 2) == bad                     # k_out inside q
    assert _norm_rope(ko=2 << 20) == bad                              # k_out on q_out
    assert _norm_rope(k=2 << 20) == bad                               # q_out on k
    # heads of one projection: q's 32 and the 8 keys right after share a span, but no byte; one head nearer they do
    fused = dict(ldq=6144, ldk=6144, ldqo=6144, qo=2 << 20)
    assert _norm_rope(k=q + 2 * 31 * 128, ko=q + 2 * 31 * 128, ldko=6144, **fused) == bad


def test_norm_rope_wrapper_refusals():
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    for call in (lambda: F.qk_norm_rope(q.float()), lambda: F.qk_norm_rope(q, q[:3]),
                 lambda: F.qk_norm_rope(q, positions=torch.zeros(4, dtype=torch.int64)),
                 lambda: F.qk_norm_rope(q, positions=torch.zeros(3, dtype=torch.int32)),
                 lambda: F.qk_norm_rope(q, q_gain=torch.ones(64, dtype=torch.bfloat16)),
                 lambda: F.qk_norm_rope(q, q_out=q[:, :4]), lambda: F.qk_norm_rope(q.transpose(0, 1)),
                 lambda: F.qk_norm_rope(q[:, ::2]), lambda: F.qk_norm_rope(q)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            call()


def test_norm_rope_oracle():
    r = np.random.default_rng(1)
    x, gain = r.normal(size=(5, 3, 128)), r.normal(size=128)
    y = O.norm_rope(x, gain, [0, 1, 2, 1000, 70000], 1e-6, 1e4)
    # position 0 only norms; rotations keep each pair's length; unit mean square without a gain
    assert np.allclose(y[0], O.rms_norm(x[0], gain, 1e-6), rtol=1e-13)
    n = O.rms_norm(x, gain, 1e-6)
    assert np.allclose(y[..., :64] ** 2 + y[..., 64:] ** 2, n[..., :64] ** 2 + n[..., 64:] ** 2, rtol=1e-11)
    assert np.allclose((O.norm_rope(x, None, np.arange(5), 0.0, 1e4) ** 2).mean(-1), 1.0, rtol=1e-12)
    # scores depend on the distance alone
    a, b = O.norm_rope(x[:1], None, [10], 0.0, 1e4), O.norm_rope(x[1:2], None, [25], 0.0, 1e4)
    c, d = O.norm_rope(x[:1], None, [110], 0.0, 1e4), O.norm_rope(x[1:2], None, [125], 0.0, 1e4)
    assert np.allclose((a * b).sum(-1), (c * d).sum(-1), rtol=1e-9)


# ---------------------------------------------------------------- eviction
def _evict(**kw):
    a = dict(codes=1 << 20, bs=12800, acc=2 << 20, acs=100, lens=None, B=3, T=100, keep=60, recent=5, G=256, levels=16,
             out=3 << 20, os=7680, acc_out=4 << 20, aos=60, lens_out=None, kept=None, ws=5 << 20, wsb=1 << 30,
             stream=None)
    a.update(kw)
    return F.cache_evict_raw(*a.values())


def test_evict_refusals():
    bad, un, mis = F.FSQ_ERR_INVALID_ARG, F.FSQ_ERR_UNSUPPORTED, F.FSQ_ERR_MISALIGNED
    assert _evict(B=0, codes=None) == F.FSQ_OK and _evict(T=0, acc=None) == F.FSQ_OK
    for kw in (dict(B=-1), dict(T=-1), dict(keep=0), dict(recent=-1), dict(recent=61), dict(codes=None),
               dict(acc=None), dict(out=None), dict(acc_out=None), dict(bs=12784), dict(acs=99), dict(os=7664),
               dict(aos=59),
               dict(out=1 << 20), dict(acc_out=2 << 20),                    # half in place
               dict(out=1 << 20, acc_out=2 << 20, aos=100),                  # in place with another stride
               dict(out=(1 << 20) + 12800), dict(acc_out=(2 << 20) + 400)):  # overlapping, not in place
        assert _evict(**kw) == bad, kw
    for kw in (dict(G=85), dict(levels=8), dict(G=578), dict(G=86, levels=4), dict(T=1 << 31, bs=1 << 40, acs=1 << 31),
               dict(keep=1 << 31, os=1 << 40, aos=1 << 31), dict(B=1 << 40)):
        assert _evict(**kw) == un, kw
    for kw in (dict(codes=(1 << 20) + 8), dict(out=(3 << 20) + 8), dict(bs=12808), dict(os=7688), dict(acc=(2 << 20) + 2),
               dict(acc_out=(4 << 20) + 1), dict(lens=2), dict(lens_out=2), dict(kept=2), dict(ws=(5 << 20) + 128)):
        assert _evict(**kw) == mis, kw
    need = F.cache_evict_workspace_size(3, 100, 256, 16)
    assert need > 0 and need % 256 == 0
    assert _evict(wsb=need - 1) == F.FSQ_ERR_WORKSPACE and _evict(ws=None) == F.FSQ_ERR_WORKSPACE
    for a in ((-1, 100, 256), (3, -1, 256), (3, 100, 85), (3, 1 << 31, 256), (1 << 40, 100, 256)):
        assert F.cache_evict_workspace_size(*a) == 0


def test_evict_wrapper_refusals():
    codes, acc = torch.zeros((2, 32, 42), dtype=torch.uint8), torch.zeros((2, 30))
    ok = dict(T=30, n_keep=10, n_recent=2, G=84)
    for call in (lambda: F.cache_evict(codes, acc.double(), **ok), lambda: F.cache_evict(codes, acc, **{**ok, "G": 80}),
                 lambda: F.cache_evict(codes, acc, **{**ok, "T": 31}), lambda: F.cache_evict(codes, acc[:1], **ok),
                 lambda: F.cache_evict(codes, acc, out=codes.clone(), **ok),
                 lambda: F.cache_evict(codes, acc, out=codes[:, :9].clone(), acc_out=acc.clone(), **ok),
                 lambda: F.cache_evict(codes, acc, kept=torch.zeros((2, 9), dtype=torch.int32), **ok),
                 lambda: F.cache_evict(codes, acc, seq_lens=torch.zeros(2, dtype=torch.int64), **ok),
                 lambda: F.cache_evict(codes[:, ::2], acc[:, :16], **{**ok, "T": 16}),
                 lambda: F.cache_evict(codes, acc, **ok)):  # the last: not on a GPU
        with pytest.raises(ValueError):
            call()


def test_evict_oracle():
    a = [3.0, 1.0, 3.0, 0.0, 5.0, 1.0, 2.0, 9.0]
    assert O.evict(a, 8, 8, 2).tolist() == list(range(8))
    assert O.evict(a, 8, 4, 2).tolist() == [0, 4, 6, 7]      # 5, then the first of the 3s; the last two stay
    assert O.evict(a, 8, 5, 2).tolist() == [0, 2, 4, 6, 7]
    assert O.evict(a, 6, 3, 3).tolist() == [3, 4, 5]
    assert O.evict(a, 7, 1, 0).tolist() == [4]
    assert O.evict([math.nan, -math.inf, -1.0, 0.0], 4, 3, 0).tolist() == [1, 2, 3]


# ---------------------------------------------------------------- shared-prefix attention, attention weights
def _prefix(**kw):
    a = dict(q=1 << 20, B=3, n_q=32, d=128, prefix=2 << 20, Tp=100, codes=3 << 20, bs=12800, T=100, G=256, W=4 << 20,
             n_kv=8, opts=F.attn_opts(), ws=5 << 20, wsb=1 << 40, o=6 << 20, stream=None)
    a.update(kw)
    return F.decode_attn_prefix_raw(*a.values())


def _weights(**kw):
    a = dict(q=1 << 20, B=3, n_q=32, d=128, codes=3 << 20, bs=12800, T=100, G=256, W=4 << 20, n_kv=8,
             opts=F.attn_opts(), acc=7 << 20, acs=100, ws=5 << 20, wsb=1 << 40, stream=None)
    a.update(kw)
    return F.attn_weights_raw(*a.values())


def test_prefix_refusals():
    bad, un, mis = F.FSQ_ERR_INVALID_ARG, F.FSQ_ERR_UNSUPPORTED, F.FSQ_ERR_MISALIGNED
    assert _prefix(B=0, q=None, prefix=None) == F.FSQ_OK
    for kw in (dict(B=-1), dict(Tp=0), dict(T=-1), dict(n_q=12), dict(n_q=0), dict(q=None), dict(prefix=None),
               dict(codes=None), dict(W=None), dict(o=None), dict(bs=12784), dict(opts=F.attn_opts(num_splits=-1)),
               dict(opts=F.attn_opts(variant=7))):
        assert _prefix(**kw) == bad, kw
    for kw in (dict(d=64), dict(G=255), dict(G=258), dict(n_q=136), dict(B=65536), dict(Tp=1 << 40),
               dict(opts=F.attn_opts(rope_knorm=True)), dict(opts=F.attn_opts(variant="expand")),
               dict(opts=F.attn_opts(variant="hybrid")), dict(opts=F.attn_opts(levels=8))):
        assert _prefix(**kw) == un, kw
    lens = F.attn_opts()
    lens.seq_lens = 18
    for kw in (dict(q=(1 << 20) + 2), dict(prefix=(2 << 20) + 8), dict(codes=(3 << 20) + 8), dict(bs=12808),
               dict(W=(4 << 20) + 2), dict(o=(6 << 20) + 4), dict(ws=(5 << 20) + 128), dict(opts=lens)):
        assert _prefix(**kw) == mis, kw
    need = F.prefix_workspace_size(3, 100, 100, 32, 8, 128, 256)
    assert need > 0 and need % 256 == 0
    assert _prefix(wsb=need - 1) == F.FSQ_ERR_WORKSPACE and _prefix(ws=None) == F.FSQ_ERR_WORKSPACE
    assert F.prefix_workspace_size(3, 0, 100, 32, 8, 128, 256) == 0
    assert F.prefix_workspace_size(3, 100, 0, 128, 8, 128, 256) > 0


def test_weights_refusals():
    bad, un, mis = F.FSQ_ERR_INVALID_ARG, F.FSQ_ERR_UNSUPPORTED, F.FSQ_ERR_MISALIGNED
    assert _weights(B=0, q=None) == F.FSQ_OK
    for kw in (dict(B=-1), dict(T=0), dict(n_q=12), dict(q=None), dict(codes=None), dict(W=None), dict(acc=None),
               dict(bs=12784), dict(acs=99), dict(opts=F.attn_opts(num_splits=-1))):
        assert _weights(**kw) == bad, kw
    for kw in (dict(d=64), dict(G=255), dict(G=578), dict(n_q=72), dict(B=65536), dict(T=1 << 40),
               dict(opts=F.attn_opts(rope_knorm=True)), dict(opts=F.attn_opts(variant="expand")),
               dict(opts=F.attn_opts(levels=8))):
        assert _weights(**kw) == un, kw
    for kw in (dict(q=(1 << 20) + 2), dict(codes=(3 << 20) + 8), dict(bs=12808), dict(W=(4 << 20) + 2),
               dict(acc=(7 << 20) + 2), dict(ws=(5 << 20) + 128)):
        assert _weights(**kw) == mis, kw
    need = F.attn_weights_workspace_size(3, 100, 32, 8, 128, 256)
    assert need > 0 and _weights(wsb=need - 1) == F.FSQ_ERR_WORKSPACE and _weights(ws=None) == F.FSQ_ERR_WORKSPACE
    for L, G in ((16, 576), (256, 576), (4, 576), (16, 2)):  # every width, up to 64 heads
        assert F.attn_weights_workspace_size(3, 100, 64, 8, 128, G, F.attn_opts(levels=L)) > 0


def test_attention_wrapper_refusals():
    q, W = torch.zeros((2, 16, 128), dtype=torch.bfloat16), torch.zeros((2048, 84), dtype=torch.bfloat16)
    codes, prefix, acc = torch.zeros((2, 32, 42), dtype=torch.uint8), torch.zeros((50, 42), dtype=torch.uint8), torch.zeros(2, 30)
    for call in (lambda: F.decode_attn_prefix(q, prefix, codes, W, 51, 30, 8, 84),
                 lambda: F.decode_attn_prefix(q, prefix, codes, W, 50, 33, 8, 84),
                 lambda: F.decode_attn_prefix(q, prefix, None, W, 50, 30, 8, 84),
                 lambda: F.decode_attn_prefix(q, prefix, codes[:1], W, 50, 30, 8, 84),
                 lambda: F.decode_attn_prefix(q, prefix, codes, W, 50, 30, 4, 84),
                 lambda: F.decode_attn_prefix(q.float(), prefix, codes, W, 50, 30, 8, 84),
                 lambda: F.decode_attn_prefix(q, prefix, codes, W, 50, 30, 8, 84, out=torch.zeros(2, 16, 128)),
                 lambda: F.decode_attn_prefix(q, prefix, codes, W, 50, 30, 8, 84),
                 lambda: F.attn_weights(q, codes, W, acc, 30, 8, 84, opts=F.attn_opts(seq_lens=torch.ones(3, dtype=torch.int32))),
                 lambda: F.attn_weights(q, codes, W, acc, 30, 8, 84, opts=F.attn_opts(seq_lens=torch.ones(2, dtype=torch.int64))),
                 lambda: F.attn_weights(q, codes, W, acc, 31, 8, 84), lambda: F.attn_weights(q, codes, W, acc.T, 30, 8, 84),
                 lambda: F.attn_weights(q, codes[:1], W, acc, 30, 8, 84),
                 lambda: F.attn_weights(q[:, :, :64], codes, W, acc, 30, 8, 84),
                 lambda: F.attn_weights(q, codes, W, acc.double(), 30, 8, 84),
                 lambda: F.attn_weights(q, codes, W, acc, 30, 8, 84)):  # the last of each: not on a GPU
        with pytest.raises(ValueError):
            call()


def test_attention_oracles():
    r = np.random.default_rng(3)
    B, n_q, n_kv, G, Tp, T = 2, 4, 2, 8, 9, 5
    prefix, codes = r.integers(0, 256, (Tp, G // 2), dtype=np.uint8), r.integers(0, 256, (B, T, G // 2), dtype=np.uint8)
    W, q = r.normal(size=(2 * n_kv * 128, G)), r.normal(size=(B, n_q, 128))
    got = O.decode_attn_prefix(q, prefix, codes, W, n_kv, G, lengths=[5, 0])
    # against torch's own attention over the concatenated rows
    for b, n in enumerate([5, 0]):
        K, V = O.reconstruct_kv(O.unpack(np.concatenate([prefix, codes[b, :n]]), G), W, n_kv, 128)
        t = lambda a: torch.from_numpy(a).repeat_interleave(2, 0)  # noqa: E731
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[b])[:, None], t(K), t(V))[:, 0]
        assert np.allclose(got[b], want.numpy(), rtol=1e-11)
    w = O.attn_weights(q, codes, W, n_kv, G, lengths=[5, 3])
    assert np.allclose(w.sum(1), n_q) and (w[1, 3:] == 0).all()
    # the weights give the attention back: sum_t w_ht v_t, one head at a time
    K, V = O.reconstruct_kv(O.unpack(codes[0], G), W, n_kv, 128)
    one = O.attn_weights(q[:1, :1], codes[:1], np.concatenate([W[:128], W[256:384]]), 1, G)
    assert np.allclose(one[0] @ V[0], O.decode_attn(q[:1], codes[:1], W, n_kv, G)[0, 0])
