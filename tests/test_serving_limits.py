"""The serving operators at the ends of what their documentation allows, on the
GPU against 64-bit references."""
import math

import numpy as np
import pytest
import torch

import fsq_latent_decode_b200 as F
from oracle import fsq_oracle as O

from cases import decoder_weights, oracle_cache

pytestmark = pytest.mark.gpu

DEV = "cuda"
LOG2E = math.log2(math.e)


def _dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


def _lens(*n):
    return torch.tensor(n, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- a wait that gives up beside a length out of range
def test_weights_that_time_out_beside_a_bad_length_add_nothing():
    """A length outside its range is clamped and recorded before any wait can give
    up; the time-out is reported all the same, and nothing is added."""
    G, T = 256, 3000
    codes = oracle_cache(2, T, G, 601)
    W, q = decoder_weights(32, 8, G, 2, 602)
    acc, ws = torch.full((2, T), 0.5, device=DEV), F.Workspace()
    a = (_dev(q), _dev(codes), _dev(W), acc, T, 8, G)
    F.attn_weights(*a, opts=F.attn_opts(seq_lens=_lens(T + 1, T), debug_stall_ns=2_000_000), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_TIMEOUT
    assert (acc == 0.5).all()
    F.attn_weights(*a, opts=F.attn_opts(seq_lens=_lens(T + 1, T)), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_ERR_INVALID_ARG
    assert np.allclose((acc.double() - 0.5).sum(1).cpu().numpy(), 32, rtol=1e-3)  # 2^-25 of 0.5 a token at most: 1e-4 of 3000


@pytest.mark.parametrize("call", ["prefix", "decode", "generic"])
def test_attention_that_times_out_beside_a_bad_length_says_so(call):
    L, G, T = (4, 320, 500) if call == "generic" else (16, 256, 500)
    codes = oracle_cache(2, T, G, 603, levels=L)
    W, q = decoder_weights(32, 8, G, 2, 604, levels=L)
    ws, out = F.Workspace(), []
    for stall in (2_000_000, 0):
        o = F.attn_opts(seq_lens=_lens(T + 1, T), debug_stall_ns=stall, levels=L)
        if call == "prefix":
            F.decode_attn_prefix(_dev(q), _dev(codes[0, :T]), _dev(codes), _dev(W), T, T, 8, G, opts=o, workspace=ws)
        else:
            F.decode_attn(_dev(q), _dev(codes), _dev(W), T, 8, G, opts=o, workspace=ws)
        out.append(F.workspace_status(ws.buf))
    assert out == [F.FSQ_ERR_TIMEOUT, F.FSQ_ERR_INVALID_ARG]


# ---------------------------------------------------------------- shared prefix: tails and sharp softmaxes
@pytest.mark.parametrize("splits", [1, 2, 0])
def test_prefix_counts_a_long_tail(splits):
    """One token far above 200000 equal ones, each 2^-25.5 of it: together 0.4 % of
    the softmax, on values seven times as large.

    Error of the pooled latent, in the units of its coordinates, with the strong
    token's weight 1 and the tail's in all t = N 2^-25.5: a split's fp16 weights
    are off by 2^-13 of its largest in all (the rule of the kernel's window), times
    the distance of the two latents; N / 16 additions on the tensor core, each
    truncated to 2^-23 of the sum so far, |z_strong| + t |z_tail|; N / 64
    additions of the weights, 2^-24 each; a score, 2^-20 of its products' size."""
    N, G, n_q = 200_000, 64, 4
    r = np.random.default_rng(7)
    strong, tail = r.integers(-1, 2, G), np.where(r.random(G) < 0.5, -7, 6)
    prefix = np.repeat(O.pack(tail[None]), N + 1, 0)
    prefix[0] = O.pack(strong[None])[0]
    W, q = decoder_weights(n_q, 1, G, 1, 8)
    Wk, Wv = (x[0] for x in O.split_wkv(W.float().numpy().astype(np.float64), 1, 128))
    q = q[:1, :1].expand(1, n_q, 128).contiguous()
    dot = float((Wk.T @ q[0, 0].double().numpy()) @ (strong - tail))
    if dot < 0:
        q, dot = -q, -dot
    scale = float(np.float32(25.5 / (LOG2E * dot)))
    w = 2.0 ** -(scale * dot * LOG2E)
    t = N * w
    want = Wv @ ((strong + t * tail) / (1 + t))
    ws = F.Workspace()
    got = F.decode_attn_prefix(_dev(q), _dev(prefix), None, _dev(W), N + 1, 0, 1, G,
                               opts=F.attn_opts(scale=scale, num_splits=splits, out_fp32=True), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    size = scale * LOG2E * float(np.abs(Wk.T @ q[0, 0].double().numpy()) @ (np.abs(strong) + np.abs(tail)))
    apart = np.abs(strong - tail)
    eps = (2.0 ** -13 + t * math.log(2) * 2.0 ** -20 * size) * apart + \
        N / 16 * 2.0 ** -23 * (np.abs(strong) + t * np.abs(tail)) + N / 64 * 2.0 ** -24 * np.abs(want).max()
    assert (np.abs(got[0].double().cpu().numpy() - want) <= np.abs(Wv) @ eps + 2.0 ** -20 * np.abs(want)).all()


@pytest.mark.parametrize("G,L", [(256, 16), (84, 16), (80, 256), (256, 256), (256, 4), (192, 16), (208, 16), (240, 256)])
@pytest.mark.parametrize("q_scale", [1.0, 8.0, 30.0])
def test_prefix_holds_sharp_scores(q_scale, G, L):
    """Scores that spread over hundreds of powers of two, in fp32 outputs, to the
    roundings that are left: the weights' fp16 (half a step, 2^-11) and flush
    (2^-25 of the largest, each), and the scores' fp32.

    A score s in log2 units is a sum of Gp / 16 steps of the tensor core, each
    truncating the products and the sum to 2^-23 of the largest partial sum M; its
    queries carry 22 bits and fp32 sums, independent over the coordinates: 2^-20 M
    is over four times their spread.  An output moves by the weights' relative
    errors times sum_t p_t |v_t - o|."""
    B, n_q, n_kv, Tp, T = 2, 16, 4, 1500, 40
    prefix = oracle_cache(1, Tp, G, 610 + G, levels=L)[0, :Tp]
    codes = oracle_cache(B, T, G, 611 + G, levels=L)
    W, q = decoder_weights(n_q, n_kv, G, B, 612, levels=L)
    q = (q.float() * q_scale).to(torch.bfloat16)
    ws = F.Workspace()
    got = F.decode_attn_prefix(_dev(q), _dev(prefix), _dev(codes), _dev(W), Tp, T, n_kv, G,
                               opts=F.attn_opts(levels=L, out_fp32=True), workspace=ws).double().cpu().numpy()
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    Wk, Wv = O.split_wkv(W.float().numpy().astype(np.float64), n_kv, 128)
    pad = -G % 16
    for b in range(B):
        z = O.unpack(np.concatenate([prefix, codes[b, :T]]), G, L).astype(np.float64)
        for h in range(n_q):
            j = h // (n_q // n_kv)
            qa = Wk[j].T @ q[b, h].double().numpy() / math.sqrt(128)
            p, v = O.softmax(z @ qa), z @ Wv[j].T
            o = p @ v
            steps = np.pad(z * qa * LOG2E, ((0, 0), (0, pad))).reshape(len(z), -1, 16).sum(-1)
            M = np.abs(np.cumsum(steps, 1)).max()
            rel = 2.0 ** -11 + math.log(2) * ((G + pad) / 16 * 2.0 ** -22 + 2.0 ** -20) * M
            away = np.abs(v - o)
            tol = rel * (p @ away) + len(z) * 2.0 ** -25 * away.max(0) + 2.0 ** -18 * (np.abs(o) + p @ np.abs(v))
            assert (np.abs(got[b, h] - o) <= tol).all(), (b, h, (np.abs(got[b, h] - o) / tol).max())


# ---------------------------------------------------------------- attention weights: a common component of W_k
@pytest.mark.parametrize("G,L,spread", [(256, 16, 0), (84, 16, 0), (576, 16, 6), (144, 256, 0), (256, 256, 0), (320, 4, 0)])
def test_weights_under_a_common_component(G, L, spread):
    """W_k with a component that all coordinates share (up to 2^-spread of it, alike in
    a pair), on latents whose coordinates cancel in pairs: it leaves the scores
    alone, but sum_g q'_g is large.

    A score's products are at most max|q'| max|z| and its partial sums that and
    max|s|: together M, to which each of its Gp / 16 steps truncates products
    and sum, 2^-23 M each.  The queries' own roundings (22 bits, fp32 sums of 128)
    are independent over the coordinates, of spread 1.3 2^-24 |q'_g| each: six
    times that over all of them.  The log-sum-exp carries the same once more."""
    T = 3000
    r = np.random.default_rng(G + L)
    top = L // 2 - 1
    z = np.empty((T, G), np.int64)
    z[:, ::2] = np.clip(np.round(r.normal(size=(T, G // 2)) * 0.58 * L / 2), -top, top)
    z[:, 1::2] = -z[:, ::2]
    codes = np.zeros((1, (T + 15) // 16 * 16, F.row_bytes(G, L)), np.uint8)
    codes[0, :T] = O.pack(z, L)
    W, q = decoder_weights(1, 1, G, 1, 13, levels=L)
    common = torch.from_numpy(8.0 * 16 / L * 2.0 ** -(spread * r.random(G // 2).repeat(2))).float()
    W[:128] = (W[:128].float() + common).to(torch.bfloat16)
    q = q.abs()
    acc, ws = torch.zeros((1, T), device=DEV), F.Workspace()
    F.attn_weights(_dev(q), _dev(codes), _dev(W), acc, T, 1, G, opts=F.attn_opts(levels=L), workspace=ws)
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    qa = W[:128].double().numpy().T @ q[0, 0].double().numpy() / math.sqrt(128) * LOG2E
    s = z @ qa
    want = O.softmax(s * math.log(2))
    big = np.abs(qa).max()
    M = big * np.abs(z).max() + np.abs(s).max()
    trunc = (G + 15) // 16 * 2.0 ** -22 * M
    rounding = 6 * math.sqrt((z * z).mean() * (qa * qa).sum()) * 1.3 * 2.0 ** -24
    got = acc[0].double().cpu().numpy()
    live = want > 1e-30
    worst = (np.abs(got - want)[live] / want[live]).max()
    assert worst <= 2 * math.log(2) * (trunc + rounding), worst
    assert (got[~live] <= 2e-30).all()


# ---------------------------------------------------------------- eviction: rows that stay whole, in clusters
@pytest.mark.parametrize("B,T", [(300, 5000), (300, 20001), (150, 70000)])
@pytest.mark.parametrize("recent", ["some", "all"])
def test_evict_of_rows_without_a_choice(B, T, recent):
    """Rows of several CTAs that select nothing, because they are short enough or
    because only recent tokens stay, in more clusters than run at once, between rows
    that do select."""
    G, keep = 4, T - 700
    n_recent = keep if recent == "all" else 100
    r = np.random.default_rng(T)
    codes = r.integers(0, 256, (B, (T + 15) // 16 * 16, 2), dtype=np.uint8)
    acc = r.exponential(size=(B, T)).astype(np.float32)
    lens = np.array([(keep, keep - 333, T, T - 1, 5)[b % 5] for b in range(B)], np.int32)
    dc, da, dl = _dev(codes), _dev(acc), _dev(lens)
    out, ao = torch.zeros((B, (keep + 15) // 16 * 16, 2), dtype=torch.uint8, device=DEV), torch.zeros((B, keep), device=DEV)
    kept, lo, ws = torch.zeros((B, keep), dtype=torch.int32, device=DEV), torch.zeros_like(dl), F.Workspace()
    want = [O.evict(acc[b], lens[b], keep, n_recent) if recent == "some" and lens[b] > keep
            else np.arange(max(0, lens[b] - keep), lens[b]) for b in range(B)]
    for _ in range(3):
        F.cache_evict(dc, da, T, keep, n_recent, G=G, seq_lens=dl, out=out, acc_out=ao, lens_out=lo, kept=kept, workspace=ws)
        assert F.workspace_status(ws.buf) == F.FSQ_OK
        got, gc, ga = kept.cpu().numpy(), out.cpu().numpy(), ao.cpu().numpy()
        assert np.array_equal(lo.cpu().numpy(), np.minimum(lens, keep))
        for b, at in enumerate(want):
            assert np.array_equal(got[b, :len(at)], at) and (got[b, len(at):] == -1).all()
            assert np.array_equal(gc[b, :len(at)], codes[b, at]) and np.array_equal(ga[b, :len(at)], acc[b, at])


# ---------------------------------------------------------------- a graph and a workspace that grows
def test_a_graph_replays_in_the_workspace_it_was_captured_with():
    """After a capture the same workspace grows for a longer call: the graph's buffer is
    not handed out to tensors made since."""
    G, T = 84, 300
    codes = oracle_cache(2, T, G, 621)
    W, q = decoder_weights(16, 8, G, 2, 622)
    a, ws = (_dev(q), _dev(codes), _dev(W)), F.Workspace()
    acc = torch.zeros((2, T), device=DEV)
    want = F.attn_weights(*a, torch.zeros_like(acc), T, 8, G, workspace=ws).clone()
    old, size = ws.buf.data_ptr(), ws.buf.numel()
    g, o = torch.cuda.CUDAGraph(), F.attn_opts()
    with torch.cuda.graph(g):
        F.attn_weights(*a, acc, T, 8, G, opts=o, workspace=ws)
    acc.zero_()
    ws.get(4 * size)
    assert ws.buf.data_ptr() != old
    fill = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(40)]
    assert all(f.data_ptr() != old for f in fill)
    g.replay()
    assert torch.equal(acc, want) and all((f == 7).all() for f in fill)
