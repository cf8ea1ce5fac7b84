"""The serving attention calls on the GPU against the fp64 oracle: rows that
share a prefix, and a run of the serving operators together.

Tolerance of the shared-prefix form (TOL, 5e-3 of the largest output, as for the
other absorbed kernels): Q' is rounded to fp16, half a step 2^-11 of each weight
at most, independently, so a score moves by 2^-11 / sqrt(3) of the root sum of
squares of its products, which is the spread of the scores, about 3 here: 8e-4
in the exponent and, relative, in the output.  P's own rounding (2^-11) averages
out over the tokens.  5e-3 is six times that; scores that spread further are
held to the floor that rounding Q' alone reaches (query_fp16_floor)."""
import math

import numpy as np
import pytest
import torch

import fsq_latent_decode_b200 as F
from oracle import fsq_oracle as O

from cases import TOL, decoder_weights, oracle_cache, padded_len, rel_err

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


def query_fp16_floor(q, rows, W_kv, n_kv, G, ref, levels=16):
    """The error, against the oracle's `ref`, of attention computed exactly except
    that each head's absorbed query is rounded to fp16 after the power of two of
    its largest weight is taken out.  rows: per batch row its packed tokens."""
    q = np.asarray(q, np.float64)
    B, n_q, d_h = q.shape
    Wk, Wv = O.split_wkv(W_kv, n_kv, d_h)
    out = np.zeros(q.shape)
    for b in range(B):
        z = O.unpack(rows[b], G, levels).astype(np.float64)
        for h in range(n_q):
            j = h // (n_q // n_kv)
            qa = (Wk[j].T @ q[b, h]) / math.sqrt(d_h) * math.log2(math.e)
            top = 2.0 ** math.floor(math.log2(np.abs(qa).max()))
            qa = (qa / top).astype(np.float16).astype(np.float64) * top
            out[b, h] = Wv[j] @ (O.softmax(z @ qa * math.log(2.0)) @ z)
    return rel_err(out, ref)


def _case(B, n_q, n_kv, G, L, Tp, T, seed, q_scale=1.0):
    prefix = oracle_cache(1, Tp, G, seed, levels=L)[0, :Tp]
    codes = oracle_cache(B, T, G, seed + 1, levels=L) if T else None
    W, q = decoder_weights(n_q, n_kv, G, B, seed + 2, levels=L)
    return prefix, codes, W, (q.float() * q_scale).to(torch.bfloat16)


def _prefix(q, prefix, codes, W, n_kv, G, T, lens=None, ws=None, **kw):
    o = F.attn_opts(seq_lens=None if lens is None else _dev(torch.tensor(lens, dtype=torch.int32)), **kw)
    ws = ws or F.Workspace()
    got = F.decode_attn_prefix(_dev(q), _dev(prefix), None if codes is None else _dev(codes), _dev(W), len(prefix), T,
                               n_kv, G, opts=o, workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    return got


def _ref(q, prefix, codes, W, n_kv, G, L, T, lens=None):
    codes = np.zeros((q.shape[0], 0, prefix.shape[1]), np.uint8) if codes is None else codes[:, :T]
    return O.decode_attn_prefix(q.float().numpy(), prefix, codes, W.float().numpy(), n_kv, G, lengths=lens, levels=L)


# widths whose rows are 16-byte pieces, and rows of 42, 60, 3, 1, 12, 5 bytes;
# grouped heads that the merge shares W_v for (1, 2, 4, 8, 16) and others (3, 5)
SHAPES = [
    (2, 16, 8, 256, 16), (3, 32, 8, 256, 16), (5, 32, 8, 84, 16), (2, 32, 8, 160, 16), (9, 16, 8, 120, 16),
    (3, 8, 2, 6, 16), (1, 4, 4, 2, 16), (33, 4, 1, 64, 16), (2, 64, 8, 96, 16), (3, 128, 8, 256, 16),
    (4, 12, 4, 44, 16), (3, 40, 8, 84, 16), (2, 48, 3, 256, 16), (7, 1, 1, 32, 16), (2, 32, 8, 256, 256),
    (4, 32, 8, 80, 256), (3, 16, 8, 144, 256), (2, 16, 8, 10, 256), (3, 32, 8, 256, 4), (2, 16, 8, 64, 4),
    (5, 16, 8, 48, 4), (2, 16, 8, 20, 4), (2, 16, 8, 4, 4),
]


@pytest.mark.parametrize("Tp,T", [(1, 1), (65, 0), (200, 33), (1000, 129)])
@pytest.mark.parametrize("B,n_q,n_kv,G,L", SHAPES)
def test_prefix_parity(B, n_q, n_kv, G, L, Tp, T):
    prefix, codes, W, q = _case(B, n_q, n_kv, G, L, Tp, T, seed=1000 + G + Tp)
    lens = None if T < 2 else [T - (b * 17) % T if b % 3 != 2 else 0 for b in range(B)]  # some rows have no own token yet
    got = _prefix(q, prefix, codes, W, n_kv, G, T, lens, levels=L, out_fp32=True).cpu().numpy()
    ref = _ref(q, prefix, codes, W, n_kv, G, L, T, lens)
    tol = max(TOL, 1.1 * query_fp16_floor(q.float().numpy(), _rows(prefix, codes, T, lens, B), W.float().numpy(), n_kv, G,
                                          ref, L))
    assert rel_err(got, ref) <= tol


def _rows(prefix, codes, T, lens, B):
    return [prefix if codes is None else np.concatenate([prefix, codes[b, :T if lens is None else lens[b]]])
            for b in range(B)]


@pytest.mark.parametrize("splits", [0, 1, 2, 7, 50, 1000])
def test_prefix_split_counts(splits):
    prefix, codes, W, q = _case(6, 32, 8, 256, 16, 3001, 300, seed=7)
    lens = [300, 1, 64, 65, 0, 299]
    got = _prefix(q, prefix, codes, W, 8, 256, 300, lens, num_splits=splits, out_fp32=True).cpu().numpy()
    assert rel_err(got, _ref(q, prefix, codes, W, 8, 256, 16, 300, lens)) <= TOL


@pytest.mark.parametrize("G,L", [(256, 16), (84, 16), (80, 256), (256, 4)])
@pytest.mark.parametrize("kind", ["flat", "sharp", "rising", "saturated", "long"])
def test_prefix_softmax_corners(kind, G, L):
    """Equal scores; a near one-hot softmax; scores that climb, so that the running
    maximum is raised again and again; codes at both ends; one split of 20k tokens."""
    n_q, n_kv, B, T = 32, 8, 4, 40
    Tp = 20000 if kind == "long" else 1500
    prefix, codes, W, q = _case(B, n_q, n_kv, G, L, Tp, T, seed=300 + G,
                                q_scale={"flat": 0.0, "sharp": 30.0, "rising": 8.0, "long": 0.05}.get(kind, 1.0))
    if kind == "rising":  # one key head and one query for all, tokens in ascending order of its score
        W = W.clone()
        W[:n_kv * 128] = W[:128].repeat(n_kv, 1)
        q = q[:1, :1].expand(B, n_q, 128).contiguous()
        s = O.unpack(prefix, G, L).astype(np.float64) @ (W[:128].double().numpy().T @ q[0, 0].double().numpy())
        prefix = prefix[np.argsort(s, kind="stable")]
    elif kind == "saturated":
        prefix, codes = prefix.copy(), codes.copy()
        prefix[::3], prefix[1::3], codes[:, ::2] = 0, 255, 255
    got = _prefix(q, prefix, codes, W, n_kv, G, T, num_splits=1 if kind == "long" else 0, levels=L,
                  out_fp32=True).cpu().numpy()
    ref = _ref(q, prefix, codes, W, n_kv, G, L, T)
    tol = TOL
    if kind in ("sharp", "rising"):
        tol = max(TOL, 1.1 * query_fp16_floor(q.float().numpy(), _rows(prefix, codes, T, None, B), W.float().numpy(), n_kv,
                                              G, ref, L))
    assert rel_err(got, ref) <= tol


def test_prefix_agrees_with_decode_of_the_whole_rows_and_bf16():
    B, n_q, n_kv, G, Tp, T = 4, 32, 8, 256, 1024, 64
    prefix, codes, W, q = _case(B, n_q, n_kv, G, 16, Tp, T, seed=11)
    whole = np.concatenate([np.repeat(prefix[None], B, 0), codes[:, :T]], 1)
    want = F.decode_attn(_dev(q), _dev(whole), _dev(W), Tp + T, n_kv, G, opts=F.attn_opts(out_fp32=True))
    got = _prefix(q, prefix, codes, W, n_kv, G, T, out_fp32=True)
    assert rel_err(got.cpu().numpy(), want.cpu().numpy()) <= TOL
    assert torch.equal(_prefix(q, prefix, codes, W, n_kv, G, T), got.to(torch.bfloat16))
    # the default scale, given by hand, and another one
    assert torch.equal(_prefix(q, prefix, codes, W, n_kv, G, T, scale=1 / math.sqrt(128), out_fp32=True), got)
    half = _prefix((q.float() * 0.5).to(torch.bfloat16), prefix, codes, W, n_kv, G, T, out_fp32=True)
    assert torch.equal(_prefix(q, prefix, codes, W, n_kv, G, T, scale=0.5 / math.sqrt(128), out_fp32=True), half)


def test_prefix_extreme_queries_stay_in_their_head():
    """Queries near the ends of bf16's range keep their precision (Q' is scaled per
    head); a query that is not finite spoils its own head alone; a query of zeros
    gives the mean."""
    B, n_q, n_kv, G, T = 3, 16, 8, 84, 20
    prefix, codes, W, q = _case(B, n_q, n_kv, G, 16, 700, T, seed=21)
    base = _prefix(q, prefix, codes, W, n_kv, G, T, out_fp32=True)
    for s in (2.0 ** 60, 2.0 ** -60):
        got = _prefix((q.float() * s).to(torch.bfloat16), prefix, codes, W, n_kv, G, T, scale=1 / math.sqrt(128) / s,
                      out_fp32=True)
        assert torch.equal(got, base)
    bad = q.clone()
    bad[1, 3, 7] = float("inf")
    bad[2, 5, 9] = float("nan")
    bad[0, 0] = 0.0
    got = _prefix(bad, prefix, codes, W, n_kv, G, T, out_fp32=True)
    assert not torch.isfinite(got[1, 3]).any() and not torch.isfinite(got[2, 5]).any()
    keep = torch.ones((B, n_q), dtype=torch.bool)
    keep[1, 3] = keep[2, 5] = keep[0, 0] = False
    assert torch.equal(got.cpu()[keep], base.cpu()[keep])
    assert rel_err(got[0, 0].cpu().numpy(), _ref(bad[:1], prefix, codes[:1], W, n_kv, G, 16, T)[0, 0]) <= TOL


def test_prefix_reads_and_writes_only_its_own():
    """Bytes behind the prefix's last token, behind a row's last own token and
    between the rows change nothing; the output's neighbours stay."""
    B, n_q, n_kv, G, Tp, T = 3, 16, 8, 84, 333, 77
    prefix, codes, W, q = _case(B, n_q, n_kv, G, 16, Tp, T, seed=31)
    lens = [77, 5, 40]
    outs = []
    for fill in (0, 255):
        long = np.full((Tp + 200, 42), fill, np.uint8)
        long[:Tp] = prefix
        wide = np.full((B, 160, 42), fill, np.uint8)
        for b in range(B):
            wide[b, :lens[b]] = codes[b, :lens[b]]
        buf = torch.full((B + 2, n_q, 128), 7.0, device=DEV)
        o = F.attn_opts(out_fp32=True, seq_lens=_dev(torch.tensor(lens, dtype=torch.int32)))
        F.decode_attn_prefix(_dev(q), _dev(long), _dev(wide), _dev(W), Tp, T, n_kv, G, opts=o, out=buf[1:-1])
        assert (buf[0] == 7).all() and (buf[-1] == 7).all()
        outs.append(buf.clone())
    assert torch.equal(*outs)


def test_prefix_out_of_range_length():
    prefix, codes, W, q = _case(3, 16, 8, 84, 16, 100, 50, seed=41)
    ws = F.Workspace()
    o = F.attn_opts(out_fp32=True, seq_lens=_dev(torch.tensor([51, -1, 50], dtype=torch.int32)))
    got = F.decode_attn_prefix(_dev(q), _dev(prefix), _dev(codes), _dev(W), 100, 50, 8, 84, opts=o, workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_INVALID_ARG
    assert rel_err(got.cpu().numpy(), _ref(q, prefix, codes, W, 8, 84, 16, 50, [50, 0, 50])) <= TOL


def test_prefix_bounded_wait_gives_up_and_next_call_recovers():
    prefix, codes, W, q = _case(4, 32, 8, 256, 16, 3000, 100, seed=51)
    a = [_dev(x) for x in (q, prefix, codes, W)]
    ws = F.Workspace()
    F.decode_attn_prefix(*a, 3000, 100, 8, 256, opts=F.attn_opts(debug_stall_ns=2_000_000), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_TIMEOUT
    got = F.decode_attn_prefix(*a, 3000, 100, 8, 256, opts=F.attn_opts(out_fp32=True), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    assert rel_err(got.cpu().numpy(), _ref(q, prefix, codes, W, 8, 256, 16, 100)) <= TOL


def test_prefix_captured_and_on_another_stream():
    prefix, codes, W, q = _case(4, 32, 8, 256, 16, 2000, 100, seed=61)
    a = [_dev(x) for x in (q, prefix, codes, W)]
    lens = _dev(torch.tensor([100, 3, 0, 64], dtype=torch.int32))
    o, out = F.attn_opts(seq_lens=lens), torch.empty((4, 32, 128), dtype=torch.bfloat16, device=DEV)
    ws = F.Workspace()

    def call(out):
        return F.decode_attn_prefix(*a, 2000, 100, 8, 256, opts=o, workspace=ws, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = call(out).clone()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    g.replay()
    assert torch.equal(out, first)
    a[0].mul_(-1)
    lens.copy_(torch.tensor([1, 100, 50, 0], dtype=torch.int32))
    g.replay()
    replayed = out.clone()
    assert torch.equal(call(torch.empty_like(out)), replayed)
    want = _ref(-q, prefix, codes, W, 8, 256, 16, 100, [1, 100, 50, 0])
    assert (np.abs(replayed.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + TOL * np.abs(want).max()).all()


# ---------------------------------------------------------------- attention weights
# Relative error of one weight, by the size of the largest score s (log2 units):
# the tensor core adds a score up in at most 36 steps (G = 576), each truncated to
# an fp32 of at most |s|, 2^-23 |s|: 36 2^-23 |s|, 6.9e-5 at 16; the log-sum-exp
# carries the same; times ln 2: 9.5e-5 in the worst case at |s| = 16.  Q' (22 bits,
# fp32 sums of 128), ex2 and the sums add below 1e-6 |s|.  So 1e-4 max(1, |s| / 16).
def _weights_case(B, n_q, n_kv, G, L, T, seed, q_scale=1.0):
    codes = oracle_cache(B, T, G, seed, levels=L)
    W, q = decoder_weights(n_q, n_kv, G, B, seed + 1, levels=L)
    return codes, W, (q.float() * q_scale).to(torch.bfloat16)


def _check_weights(q, codes, W, n_kv, G, L, T, lens=None, **kw):
    B, n_q = q.shape[:2]
    r = np.random.default_rng(T + G)
    acc0 = (r.exponential(size=(B, T + 5)) * n_q / T).astype(np.float32)
    acc0[:, ::4] = 0.0
    acc = _dev(acc0)
    ws = F.Workspace()
    o = F.attn_opts(seq_lens=None if lens is None else _dev(torch.tensor(lens, dtype=torch.int32)), levels=L, **kw)
    got = F.attn_weights(_dev(q), _dev(codes), _dev(W), acc, T, n_kv, G, opts=o, workspace=ws)
    assert got.data_ptr() == acc.data_ptr() and F.workspace_status(ws.buf) == F.FSQ_OK
    w = O.attn_weights(q.float().numpy(), codes[:, :T], W.float().numpy(), n_kv, G, lengths=lens, levels=L)
    top = 0.0
    Wk, _ = O.split_wkv(W.float().numpy(), n_kv, 128)
    for b in range(B):
        z = O.unpack(codes[b, :T], G, L).astype(np.float64)
        for h in range(n_q):
            top = max(top, np.abs(z @ (Wk[h // (n_q // n_kv)].T @ q[b, h].double().numpy())).max() / math.sqrt(128) * 1.4427)
    got = got.double().cpu().numpy()
    n = [T] * B if lens is None else lens
    for b in range(B):
        assert np.array_equal(got[b, n[b]:], acc0[b, n[b]:])  # behind the last token nothing moves
        ref = w[b, :n[b]] + acc0[b, :n[b]]
        # the last addition rounds once more
        assert (np.abs(got[b, :n[b]] - ref) <= 1e-4 * max(1.0, top / 16) * w[b, :n[b]] + 2.0 ** -23 * ref + 1e-37).all()


W_SHAPES = [(2, 16, 8, 256, 16), (3, 32, 8, 256, 16), (5, 32, 8, 84, 16), (2, 64, 8, 160, 16), (2, 8, 8, 288, 16),
            (3, 1, 1, 6, 16), (2, 12, 4, 44, 16), (2, 40, 8, 576, 16), (1, 64, 8, 576, 16), (2, 24, 3, 96, 16),
            (3, 32, 8, 80, 256), (2, 16, 8, 256, 256), (2, 48, 8, 144, 256), (1, 64, 4, 576, 256), (2, 16, 8, 10, 256),
            (2, 16, 8, 560, 256), (3, 32, 8, 320, 4), (2, 32, 8, 576, 4), (2, 16, 8, 64, 4), (2, 16, 8, 4, 4),
            (2, 16, 8, 20, 4)]


@pytest.mark.parametrize("T", [1, 128, 300, 1111])
@pytest.mark.parametrize("B,n_q,n_kv,G,L", W_SHAPES)
def test_weights_parity(B, n_q, n_kv, G, L, T):
    codes, W, q = _weights_case(B, n_q, n_kv, G, L, T, seed=500 + G + T)
    lens = None if T < 300 else [max(1, T - 256 * b - 43 * (b > 0)) for b in range(B)]
    _check_weights(q, codes, W, n_kv, G, L, T, lens)


@pytest.mark.parametrize("splits", [0, 1, 2, 9, 1000])
def test_weights_split_counts(splits):
    codes, W, q = _weights_case(3, 32, 8, 256, 16, 4000, seed=71)
    _check_weights(q, codes, W, 8, 256, 16, 4000, [4000, 1, 2049], num_splits=splits)


@pytest.mark.parametrize("G,L", [(256, 16), (84, 16), (144, 256), (320, 4)])
@pytest.mark.parametrize("q_scale", [0.0, 5.0, 60.0])
def test_weights_softmax_corners(q_scale, G, L):
    """Equal scores; sharp ones; ones that spread over thousands of powers of two,
    so that the first token's score is far below the largest."""
    codes, W, q = _weights_case(2, 32, 8, G, L, 1500, seed=80 + G, q_scale=q_scale)
    _check_weights(q, codes, W, 8, G, L, 1500, num_splits=2)


def test_weights_of_many_rows_and_a_long_row():
    codes, W, q = _weights_case(200, 16, 8, 84, 16, 200, seed=90)
    _check_weights(q, codes, W, 8, 84, 16, 200)
    codes, W, q = _weights_case(1, 16, 8, 256, 16, 40000, seed=91)
    _check_weights(q, codes, W, 8, 256, 16, 40000)


def test_weights_accumulate_over_steps_and_ignore_what_lies_behind():
    """Several steps on one workspace add up; bytes behind a row's length change nothing."""
    B, T, G = 2, 700, 84
    codes, W, q = _weights_case(B, 32, 8, G, 16, T, seed=95)
    lens = [700, 333]
    outs = []
    for fill in (0, 255):
        c = codes.copy()
        c[1, 333:] = fill
        acc, ws = torch.zeros((B, T), device=DEV), F.Workspace()
        o = F.attn_opts(seq_lens=_dev(torch.tensor(lens, dtype=torch.int32)))
        for step in range(3):
            F.attn_weights(_dev(torch.roll(q, step, 1)), _dev(c), _dev(W), acc, T, 8, G, opts=o, workspace=ws)
        outs.append(acc)
    assert torch.equal(*outs)
    total = outs[0].double().sum(1).cpu().numpy()
    assert np.allclose(total, 3 * 32, rtol=1e-5)  # every head of every step spends a weight of 1


def test_weights_bounded_wait_adds_nothing_and_next_call_recovers():
    codes, W, q = _weights_case(2, 32, 8, 256, 16, 3000, seed=97)
    acc, ws = torch.zeros((2, 3000), device=DEV), F.Workspace()
    a = (_dev(q), _dev(codes), _dev(W), acc, 3000, 8, 256)
    F.attn_weights(*a, opts=F.attn_opts(debug_stall_ns=2_000_000), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_TIMEOUT and (acc == 0).all()
    F.attn_weights(*a, workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    assert np.allclose(acc.double().sum(1).cpu().numpy(), 32, rtol=1e-5)


def test_weights_out_of_range_length_and_non_finite_queries():
    codes, W, q = _weights_case(4, 16, 8, 84, 16, 300, seed=98)
    q[3, 2, 1] = float("nan")
    acc, ws = torch.zeros((4, 300), device=DEV), F.Workspace()
    o = F.attn_opts(seq_lens=_dev(torch.tensor([301, 0, 299, 300], dtype=torch.int32)))
    F.attn_weights(_dev(q), _dev(codes), _dev(W), acc, 300, 8, 84, opts=o, workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_INVALID_ARG
    want = O.attn_weights(q[:3].float().numpy(), codes[:3, :300], W.float().numpy(), 8, 84, lengths=[300, 1, 299])
    assert np.allclose(acc[:3].cpu().numpy(), want, rtol=1e-4, atol=1e-37)
    assert torch.isnan(acc[3]).all()  # the row's sum over heads


def test_weights_captured_and_on_another_stream():
    codes, W, q = _weights_case(3, 32, 8, 256, 16, 1000, seed=99)
    a = [_dev(x) for x in (q, codes, W)]
    ws, acc = F.Workspace(), torch.zeros((3, 1000), device=DEV)
    want = F.attn_weights(*a, torch.zeros_like(acc), 1000, 8, 256, workspace=ws).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        F.attn_weights(*a, acc, 1000, 8, 256, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(acc, want)
    acc.zero_()
    g = torch.cuda.CUDAGraph()
    o = F.attn_opts()
    with torch.cuda.graph(g):
        F.attn_weights(*a, acc, 1000, 8, 256, opts=o, workspace=ws)
    acc.zero_()
    g.replay()
    assert torch.equal(acc, want)
    g.replay()
    assert torch.equal(acc, want + want)


# ---------------------------------------------------------------- the operators together
def test_serving_run():
    """A batch on one prompt: decode steps on the shared prefix with queries normed
    and rotated in place, then the rows' caches put together, weights gathered over
    steps, the caches cut to a budget in place, and decoding goes on in them."""
    B, n_q, n_kv, G, C, Tp, T = 3, 32, 8, 256, 1024, 500, 6
    r = np.random.default_rng(0)
    bf = lambda a: torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)  # noqa: E731
    prefix = oracle_cache(1, Tp, G, 77)[0, :Tp]
    W, _ = decoder_weights(n_q, n_kv, G, B, 78)
    E = bf(r.normal(size=(G, C)) * 2 / math.sqrt(C))
    gain = bf(1 + 0.1 * r.normal(size=128))
    own = torch.zeros((B, 16, 128), dtype=torch.uint8, device=DEV)
    ws = F.Workspace()
    dp, dW = _dev(prefix), _dev(W)
    for t in range(T):  # every step appends a token to each row and attends
        F.append_rows(_dev(bf(r.normal(size=(B, C)))), _dev(E), own, t)
        q = bf(r.normal(size=(B, n_q, 128)))
        dq = _dev(q)
        pos = torch.full((B,), Tp + t + 1, dtype=torch.int32, device=DEV)
        F.qk_norm_rope(dq, q_gain=_dev(gain), positions=pos, pos0=-1, q_out=dq)
        got = F.decode_attn_prefix(dq, dp, own, dW, Tp, t + 1, n_kv, G, opts=F.attn_opts(out_fp32=True), workspace=ws)
        want = _ref(dq.cpu(), prefix, own.cpu().numpy(), W, n_kv, G, 16, t + 1)
        assert rel_err(got.cpu().numpy(), want) <= TOL
    n = Tp + T
    cache = torch.zeros((B, 512, 128), dtype=torch.uint8, device=DEV)
    cache[:, :Tp], cache[:, Tp:n] = dp, own[:, :T]
    acc, lens = torch.zeros((B, 512), device=DEV), torch.tensor([n, n - 7, n - 100], dtype=torch.int32, device=DEV)
    ref, before = np.zeros((B, 512)), cache.cpu().numpy()
    for _ in range(4):
        q = bf(r.normal(size=(B, n_q, 128)))
        F.attn_weights(_dev(q), cache, dW, acc, n, n_kv, G, opts=F.attn_opts(seq_lens=lens), workspace=ws)
        ref[:, :n] += O.attn_weights(q.float().numpy(), before[:, :n], W.float().numpy(), n_kv, G, lengths=lens.tolist())
    assert np.allclose(acc.cpu().numpy(), ref, rtol=2e-4, atol=1e-30)
    keep = 410
    a = acc.cpu().numpy()
    kept = torch.empty((B, keep), dtype=torch.int32, device=DEV)
    F.cache_evict(cache, acc, n, keep, 32, G=G, seq_lens=lens, lens_out=lens, kept=kept, workspace=ws)
    rows = []
    for b, old in enumerate([n, n - 7, n - 100]):
        at = O.evict(a[b], old, keep, 32)
        assert kept[b, :len(at)].tolist() == at.tolist()
        rows.append(before[b, at])
    assert lens.tolist() == [410, 410, 406]
    assert (acc[:2, keep:] == 0).all()
    q = bf(r.normal(size=(B, n_q, 128)))
    got = F.decode_attn(_dev(q), cache, dW, keep, n_kv, G, opts=F.attn_opts(out_fp32=True, seq_lens=lens), workspace=ws)
    want = np.concatenate([O.decode_attn(q[b:b + 1].float().numpy(), rows[b][None], W.float().numpy(), n_kv, G)
                           for b in range(B)])
    assert rel_err(got.cpu().numpy(), want) <= TOL
    # the keys that the hybrid form rebuilds are normed and rotated by their place in the cut cache
    o = F.attn_opts(variant="hybrid", rope_knorm=True, out_fp32=True, seq_lens=lens)
    dq = F.qk_norm_rope(_dev(q), positions=lens, pos0=-1)
    got = F.decode_attn(dq, cache, dW, keep, n_kv, G, opts=o, workspace=ws)
    rk = dict(gain=np.ones(128), eps=1e-6, base=1e6)
    want = np.concatenate([O.decode_attn(dq[b:b + 1].float().cpu().numpy(), rows[b][None], W.float().numpy(), n_kv, G,
                                         rope_knorm=rk) for b in range(B)])
    assert rel_err(got.cpu().numpy(), want) <= TOL


def test_results_on_a_given_stream_outlive_later_allocations():
    """stream=: what a wrapper allocates belongs to that stream, so tensors made
    meanwhile on the current one do not land in a workspace that is in use."""
    B, n_q, n_kv, G, Tp, T = 2, 16, 8, 256, 300, 100
    prefix, codes, W, q = _case(B, n_q, n_kv, G, 16, Tp, T, 5)
    dq, dp, dc, dW = _dev(q), _dev(prefix), _dev(codes), _dev(W)
    acc = torch.zeros((B, T), device=DEV)

    def calls(stream):
        x = F.qk_norm_rope(dq, stream=stream)
        o = F.decode_attn_prefix(x, dp, dc, dW, Tp, T, n_kv, G, stream=stream)
        a = F.attn_weights(x, dc, dW, acc, T, n_kv, G, stream=stream)
        return x, o, a

    want = [t.clone() for t in calls(None)]
    acc.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # about 10 ms: the calls queue behind it
    got = calls(s)
    fill = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (256, 2048, 8192, 65536, 1 << 18, 1 << 20, 4 << 20)
            for _ in range(4)]
    s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    del fill
