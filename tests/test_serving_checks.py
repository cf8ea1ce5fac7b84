"""Host-side checks of the serving operators, no GPU: what a kernel's source must
order, and what the wrappers refuse and why."""
import os
import re

import pytest
import torch

import fsq_latent_decode_b200 as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_evict_select_waits_for_its_cluster_before_remote_shared_memory():
    """A cluster's CTAs may touch one another's shared memory only after a barrier of
    the whole cluster.  The first one stands before the first remote access on every
    path: outside every block of the kernel's body."""
    src = open(os.path.join(ROOT, "fsq_latent_decode_b200", "csrc", "evict.cu")).read()
    body = src[src.index("evict_select(SelectParams p, int per) {"):]
    body = re.sub(r"//[^\n]*", "", body[body.index("{"):])
    arrive, wait = body.index("cl.barrier_arrive()"), body.index("cl.barrier_wait()")
    remote = body.index("map_shared_rank")
    assert arrive < wait < remote
    for at in (arrive, wait):
        assert body[:at].count("{") - body[:at].count("}") == 1
        assert re.search(r"if \(CS > 1\) $", body[:at])


# ---------------------------------------------------------------- refusals of the wrappers, each for its own reason
# CPU tensors reach every check but the last, whose message is another one: a case
# passes only if the check that it names is there.
BF16 = torch.bfloat16
I32 = torch.int32
ELSEWHERE = "every tensor must be on the current CUDA device"


def _refused(cases):
    for match, call in cases:
        with pytest.raises(ValueError, match=re.escape(match)):
            call()


def test_norm_rope_refuses_each_argument_by_name():
    q, k = torch.zeros((4, 8, 128), dtype=BF16), torch.zeros((4, 2, 128), dtype=BF16)
    n = F.qk_norm_rope
    _refused([
        ("q must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q[0])),
        ("q must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q.transpose(0, 1))),
        ("q must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q[:, ::2])),
        ("q must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q.transpose(1, 2))),
        ("q must be [n_tok, heads, d_h] with contiguous heads", lambda: n(torch.zeros((4, 1, 256), dtype=BF16)[:, :, ::2])),
        ("q must be torch.bfloat16", lambda: n(q.float())),
        ("q must be torch.bfloat16", lambda: n(q.half())),
        ("q_out must be torch.bfloat16 of q's shape", lambda: n(q, q_out=q[:, :4])),
        ("q_out must be torch.bfloat16 of q's shape", lambda: n(q, q_out=q[:3])),
        ("q_out must be torch.bfloat16 of q's shape", lambda: n(q, q_out=q.float())),
        ("q_out must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q, q_out=torch.zeros((4, 16, 128), dtype=BF16)[:, ::2])),
        ("k must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q, k.transpose(0, 1))),
        ("k must be torch.bfloat16 [n_tok, n_k, d_h]", lambda: n(q, k[:3])),
        ("k must be torch.bfloat16 [n_tok, n_k, d_h]", lambda: n(q, k.float())),
        ("k must be torch.bfloat16 [n_tok, n_k, d_h]", lambda: n(q, torch.zeros((4, 2, 64), dtype=BF16))),
        ("k_out must be torch.bfloat16 of k's shape", lambda: n(q, k, k_out=k[:, :1])),
        ("k_out must be torch.bfloat16 of k's shape", lambda: n(q, k, k_out=k.float())),
        ("k_out must be [n_tok, heads, d_h] with contiguous heads", lambda: n(q, k, k_out=q[:, ::4])),
        ("positions must hold 4 contiguous torch.int32 values", lambda: n(q, positions=torch.zeros(4, dtype=torch.int64))),
        ("positions must hold 4 contiguous torch.int32 values", lambda: n(q, positions=torch.zeros(3, dtype=I32))),
        ("positions must hold 4 contiguous torch.int32 values", lambda: n(q, positions=torch.zeros(8, dtype=I32)[::2])),
        ("q_gain must hold 128 contiguous torch.bfloat16 values", lambda: n(q, q_gain=torch.ones(64, dtype=BF16))),
        ("q_gain must hold 128 contiguous torch.bfloat16 values", lambda: n(q, q_gain=torch.ones(128))),
        ("k_gain must hold 128 contiguous torch.bfloat16 values", lambda: n(q, k, k_gain=torch.ones(129, dtype=BF16))),
        (ELSEWHERE, lambda: n(q)),
        (ELSEWHERE, lambda: n(q, k)),
    ])


def test_evict_refuses_each_argument_by_name():
    codes, acc = torch.zeros((2, 32, 42), dtype=torch.uint8), torch.zeros((2, 30))
    ok = dict(T=30, n_keep=10, n_recent=2, G=84)
    e = lambda c=codes, a=acc, **kw: lambda: F.cache_evict(c, a, **{**ok, **kw})  # noqa: E731
    codes_is, acc_is = "codes must be uint8 [2, at least 30, 42] with contiguous rows", "acc must be fp32 [2, at least 30] with contiguous rows"
    small, few = torch.zeros((2, 16, 42), dtype=torch.uint8), torch.zeros((2, 10))
    _refused([
        (codes_is, e(codes.to(torch.int8))), ("codes must be uint8 [32, at least 30, 42] with contiguous rows", e(codes[0])), (codes_is, e(codes[:, :29])),
        (codes_is, e(torch.zeros((2, 64, 42), dtype=torch.uint8)[:, ::2])),
        (codes_is, e(torch.zeros((2, 32, 43), dtype=torch.uint8)[:, :, :42])),
        ("codes must be uint8 [2, at least 1, 42] with contiguous rows",
         e(torch.zeros((2, 1, 84), dtype=torch.uint8)[:, :, ::2], T=1, n_keep=1, n_recent=0)),
        ("codes must be uint8 [2, at least 30, 40] with contiguous rows", e(G=80)),
        ("codes must be uint8 [2, at least 33, 42] with contiguous rows", e(T=33)),
        (acc_is, e(a=acc.double())), (acc_is, e(a=acc[:1])), (acc_is, e(a=acc[:, :29])), (acc_is, e(a=acc[0])), (acc_is, e(a=acc[:, :, None])),
        (acc_is, e(a=torch.zeros((2, 60))[:, ::2])),
        ("acc must be fp32 [2, at least 31] with contiguous rows", e(T=31)),
        ("out and acc_out go together", e(out=small)), ("out and acc_out go together", e(acc_out=few)),
        ("out must be uint8 [2, at least 10, 42]", e(out=small[:, :9], acc_out=few)),
        ("out must be uint8 [2, at least 10, 42]", e(out=small[:1], acc_out=few)),
        ("acc_out must be fp32 [2, at least 10]", e(out=small, acc_out=few[:, :9])),
        ("acc_out must be fp32 [2, at least 10]", e(out=small, acc_out=few.half())),
        ("seq_lens must hold 2 contiguous torch.int32 values", e(seq_lens=torch.zeros(2, dtype=torch.int64))),
        ("seq_lens must hold 2 contiguous torch.int32 values", e(seq_lens=torch.zeros(1, dtype=I32))),
        ("lens_out must hold 2 contiguous torch.int32 values", e(lens_out=torch.zeros(3, dtype=I32))),
        ("lens_out must hold 2 contiguous torch.int32 values", e(lens_out=torch.zeros(2))),
        ("kept must hold 20 contiguous torch.int32 values", e(kept=torch.zeros((2, 9), dtype=I32))),
        ("kept must hold 20 contiguous torch.int32 values", e(kept=torch.zeros((2, 20), dtype=I32)[:, ::2])),
        (ELSEWHERE, e()), (ELSEWHERE, e(out=small, acc_out=few)),
    ])


def test_attention_calls_refuse_each_argument_by_name():
    q, W = torch.zeros((2, 16, 128), dtype=BF16), torch.zeros((2048, 84), dtype=BF16)
    codes, prefix = torch.zeros((2, 32, 42), dtype=torch.uint8), torch.zeros((50, 42), dtype=torch.uint8)
    acc = torch.zeros(2, 30)

    def p(q=q, prefix=prefix, codes=codes, W=W, Tp=50, T=30, n_kv=8, G=84, **kw):
        return lambda: F.decode_attn_prefix(q, prefix, codes, W, Tp, T, n_kv, G, **kw)

    def w(q=q, codes=codes, W=W, acc=acc, T=30, n_kv=8, G=84, **kw):
        return lambda: F.attn_weights(q, codes, W, acc, T, n_kv, G, **kw)

    q_is, W_is = "q must be contiguous torch.bfloat16 [B, n_q, d_h]", "W_kv must be contiguous torch.bfloat16 [2 * n_kv * d_h, G]"
    lens_is = "opts.seq_lens must hold 2 contiguous torch.int32 values"
    codes_is = "codes must be uint8 [2, at least 30, 42] with contiguous rows"
    for f in (p, w):
        _refused([
            (q_is, f(q=q.float())), (q_is, f(q=q[0])), (q_is, f(q=q[:, ::2])), (q_is, f(q=q.transpose(0, 1))),
            (W_is, f(W=W.float())), (W_is, f(W=W[:1024])), (W_is, f(W=W[:, :42])), (W_is, f(n_kv=4)),
            (W_is, f(W=torch.zeros((2048, 168), dtype=BF16)[:, ::2])), (W_is, f(q=q[:, :, :64].contiguous())),
            (lens_is, f(opts=F.attn_opts(seq_lens=torch.ones(3, dtype=I32)))),
            (lens_is, f(opts=F.attn_opts(seq_lens=torch.ones(2, dtype=torch.int64)))),
            (lens_is, f(opts=F.attn_opts(seq_lens=torch.ones(4, dtype=I32)[::2]))),
            (codes_is, f(codes=codes[:1])), (codes_is, f(codes=codes[:, :29])), (codes_is, f(codes=codes.int())),
            (codes_is, f(codes=codes[:, :, :41])), (codes_is, f(codes=codes[0])),
            ("codes must be uint8 [2, at least 33, 42] with contiguous rows", f(T=33, acc=torch.zeros(2, 33)) if f is w else f(T=33)),
            (ELSEWHERE, f()),
        ])
    prefix_is = "prefix must be contiguous uint8 [at least 50, 42]"
    out_is = "out must be contiguous [B, n_q, d_h] torch.bfloat16"
    acc_is = "acc must be fp32 [2, at least 30] with contiguous rows"
    _refused([
        ("prefix must be contiguous uint8 [at least 51, 42]", p(Tp=51)), (prefix_is, p(prefix=prefix[:49])),
        (prefix_is, p(prefix=prefix.int())), (prefix_is, p(prefix=prefix[:, :41])), (prefix_is, p(prefix=prefix[None])),
        (prefix_is, p(prefix=prefix[:, :, None])), (prefix_is, p(prefix=torch.zeros((50, 43), dtype=torch.uint8))),
        (prefix_is, p(prefix=torch.zeros((100, 42), dtype=torch.uint8)[::2])),
        ("codes must hold the own tokens of every row", p(codes=None)),
        (out_is, p(out=torch.zeros(2, 16, 128))), (out_is, p(out=q[:1])), (out_is, p(out=torch.zeros((2, 32, 128), dtype=BF16)[:, ::2])),
        ("out must be contiguous [B, n_q, d_h] torch.float32", p(out=torch.zeros_like(q), opts=F.attn_opts(out_fp32=True))),
        (ELSEWHERE, p(codes=None, T=0)),
        (acc_is, w(acc=acc.double())), (acc_is, w(acc=acc.T)), (acc_is, w(acc=acc[:1])), (acc_is, w(acc=acc[:, :29])),
        (acc_is, w(acc=torch.zeros(2, 60)[:, ::2])),
    ])


class _On:
    """Stands for a tensor, or with `device` for a stream, of a device of that number."""

    def __init__(self, n):
        self.n, self.device, self.cuda_stream = n, torch.device("cuda", n) if n >= 0 else torch.device("cpu"), 7

    def get_device(self):
        return self.n


def test_a_call_runs_on_the_current_device_alone(monkeypatch):
    from fsq_latent_decode_b200 import _abi
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert _abi._launch("op", _On(1), _On(1), None, _On(1)) == 7
    _refused([
        (ELSEWHERE, lambda: _abi._launch("op", None, _On(0))),           # not the current one
        (ELSEWHERE, lambda: _abi._launch("op", None, _On(1), _On(0))),   # two devices
        (ELSEWHERE, lambda: _abi._launch("op", None, _On(-1))),          # none
        ("the stream must be on the tensors' device", lambda: _abi._launch("op", _On(0), _On(1))),
    ])


def test_a_workspace_of_another_device_is_refused():
    from fsq_latent_decode_b200 import _abi
    assert _abi._scratch("op", None, torch.zeros(1), 1000).numel() == 1000
    with pytest.raises(ValueError, match="op: the workspace must be on the tensors' device, got cpu"):
        _abi._scratch("op", F.Workspace("cpu"), _On(1), 1000)


def test_a_workspace_keeps_what_a_graph_was_captured_with(monkeypatch):
    ws, capturing = F.Workspace("cpu"), False
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    import weakref
    first = weakref.ref(ws.get(1000))
    assert ws.get(900) is first()
    second = weakref.ref(ws.get(2000))
    assert first() is None  # no graph: an outgrown buffer goes
    capturing = True
    assert ws.get(500) is second()
    capturing = False
    third = weakref.ref(ws.get(5000))
    assert second() is not None and third() is not second()
    ws.get(9000)
    assert second() is not None and third() is None
    del ws
    assert second() is None


def test_evict_refuses_lengths_and_indices_that_overlap():
    """Rows read their length and write the new one at different times: the two arrays
    are one, or apart; so are the kept indices."""
    def call(lens=None, lens_out=None, kept=None, keep=60, recent=5):
        return F.cache_evict_raw(1 << 20, 12800, 2 << 20, 100, lens, 3, 100, keep, recent, 256, 16, 3 << 20, 7680, 4 << 20,
                                 60, lens_out, kept, None, 0, None)

    bad, ok = F.FSQ_ERR_INVALID_ARG, F.FSQ_ERR_WORKSPACE  # past the checks: no workspace
    m = 6 << 20
    assert call(m, m) == call(m, m + 12) == call(m, None, m + 12) == call(m, m, m + 12) == call(None, m, m + 12) == ok
    assert call(m, m + 4) == call(m + 8, m) == bad
    assert call(m, None, m) == call(m, None, m - 716) == call(None, m, m - 4) == call(m, m + 12, m + 20) == bad
    assert call(m, None, m - 720) == ok


def test_prefix_splits_hold_2_to_22_tokens_at_most():
    one = F.attn_opts(num_splits=1)
    size = lambda Tp: F.prefix_workspace_size(1, Tp, 0, 8, 2, 128, 64, one)  # noqa: E731
    assert size(1) == size(1 << 22) < size((1 << 22) + 1) == size(1 << 23) < size((1 << 23) + 1)
