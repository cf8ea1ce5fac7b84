"""The serving operators around the code cache on the GPU, against the fp64
oracle: head norms with rotary positions, eviction by accumulated weight."""
import numpy as np
import pytest
import torch

import fsq_latent_decode_b200 as F
from oracle import fsq_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _rng(*parts):
    return np.random.default_rng(list(parts))


# ---------------------------------------------------------------- head norms + rotary positions
# Error of one output (a cos - b sin or a sin + b cos), a and b the normed pair:
# one rounding to bf16 (half a step, 2^-8 of the value), and in fp32, relative to
# |a| + |b|: the sum of 128 squares (7 adds deep and a product, halved by the
# root) 5, rsqrt 2, two products 2, the rotation 3, sincospi of an angle rounded
# to 24 bits (pi 2^-25 and 2 ulp) 5: 17 roundings of 2^-24, below 2^-19.
def _norm_rope_close(got, x, gain, pos, eps, base):
    ref = O.norm_rope(x, gain, pos, eps, base)
    y = np.abs(O.rms_norm(x, np.ones(128) if gain is None else gain, eps))
    pair = np.tile(y[..., :64] + y[..., 64:], 2)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * pair).all()


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("n,n_q,n_k", [(1, 32, 8), (1, 1, 0), (2, 16, 8), (7, 5, 3), (129, 32, 8), (1183, 3, 1),
                                       (1184, 16, 8), (1189, 7, 0), (2000, 1, 2)])
@pytest.mark.parametrize("base", [1.0e4, 1.0e6])
def test_norm_rope(n, n_q, n_k, base):
    r = _rng(n, n_q, n_k)
    q, k = _bf16(r.normal(size=(n, n_q, 128)) * 3), _bf16(r.normal(size=(n, n_k, 128)))
    gq, gk = _bf16(1 + 0.3 * r.normal(size=128)), _bf16(1 + 0.3 * r.normal(size=128))
    pos = torch.from_numpy(r.integers(0, 1 << 20, n).astype(np.int32))
    if n_k:
        a, b = F.qk_norm_rope(q.to(DEV), k.to(DEV), gq.to(DEV), gk.to(DEV), positions=pos.to(DEV), rope_base=base)
        _norm_rope_close(_f64(b), _f64(k), _f64(gk), pos.numpy(), 1e-6, base)
    else:
        a = F.qk_norm_rope(q.to(DEV), q_gain=gq.to(DEV), positions=pos.to(DEV), rope_base=base)
    _norm_rope_close(_f64(a), _f64(q), _f64(gq), pos.numpy(), 1e-6, base)


@pytest.mark.parametrize("n", [3, 1500])
def test_norm_rope_of_a_fused_projection_in_place(n):
    """q and k are views of one projection, normed in place; v is left alone.
    Positions count up from a far offset, beyond 32 bits with the offset added."""
    r = _rng(n)
    qkv = _bf16(r.normal(size=(n, 48, 128)))
    x = qkv.to(DEV)
    pos0 = (1 << 33) + 5
    q, k = F.qk_norm_rope(x[:, :32], x[:, 32:40], pos0=pos0, eps=0.0, q_out=x[:, :32], k_out=x[:, 32:40])
    assert q.data_ptr() == x.data_ptr()
    pos = pos0 + np.arange(n)
    # at 2^33 the oracle's own angle (one product in 64 bits) is good to 2^33 2^-53: 2^-20, added to the bound
    ref_q = O.norm_rope(_f64(qkv[:, :32]), None, pos, 0.0, 1e6)
    got = _f64(x)
    assert (np.abs(got[:, :32] - ref_q) <= 2.0 ** -8 * np.abs(ref_q) + 2.0 ** -16).all()
    assert torch.equal(x[:, 40:].cpu(), qkv[:, 40:])
    y = qkv.to(DEV)
    z = F.qk_norm_rope(y[:, :32], y[:, 32:40], pos0=pos0, eps=0.0)
    assert torch.equal(z[0], q) and torch.equal(z[1], k)  # out of place: the same


def test_norm_rope_decode_positions_and_odd_values():
    """seq_lens with pos0 = -1 (a decode step); zero rows, huge and tiny rows,
    an infinity stays in its own head."""
    r = _rng(5)
    q = _bf16(r.normal(size=(6, 4, 128)))
    q[0, 0] = 0
    q[1, 1] *= 2.0 ** 60
    q[2, 2] *= 2.0 ** -60
    lens = torch.tensor([1, 2, 300, 40000, 7, 1], dtype=torch.int32)
    got = F.qk_norm_rope(q.to(DEV), positions=lens.to(DEV), pos0=-1)
    _norm_rope_close(_f64(got), _f64(q), None, lens.numpy() - 1, 1e-6, 1e6)
    assert (got[0, 0] == 0).all()
    bad = q.clone()
    bad[3, 1, 5] = float("inf")
    out = F.qk_norm_rope(bad.to(DEV), positions=lens.to(DEV), pos0=-1)
    same = torch.ones(6, 4, dtype=torch.bool)
    same[3, 1] = False
    assert torch.equal(out.cpu()[same], got.cpu()[same]) and not torch.isfinite(out[3, 1].float()).all()


def test_norm_rope_streams_and_graph():
    r = _rng(6)
    q = _bf16(r.normal(size=(40, 8, 128))).to(DEV)
    want = F.qk_norm_rope(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = F.qk_norm_rope(q)
    other = F.qk_norm_rope(q, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.qk_norm_rope(q, q_out=out)
    q.copy_(q * 2 + 1)
    g.replay()
    assert torch.equal(out, F.qk_norm_rope(q))


# ---------------------------------------------------------------- eviction
def _weights(kind, B, T, r):
    a = r.exponential(size=(B, T)).astype(np.float32) ** 3
    if kind == "ties":
        a = np.floor(a).astype(np.float32)      # half of them 0, long runs of equal values
    elif kind == "equal":
        a[:] = 0.25
    elif kind == "signs":
        a = r.normal(size=(B, T)).astype(np.float32)
        a[:, ::3] = 0.0
        a[:, 1::3] = np.where(r.random((B, a[:, 1::3].shape[1])) < 0.5, -0.0, a[:, 1::3])
        a[:, 4::7] = np.nan
        a[:, 5::11] = np.inf
        a[:, 6::13] = -np.inf
    return a


def _evict_case(B, T, G, levels, keep, recent, lens, kind, in_place, seed=0):
    r = _rng(B, T, G, keep, recent, seed)
    R = F.row_bytes(G, levels)
    Tm = (T + 15) // 16 * 16
    codes = r.integers(0, 256, (B, Tm, R), dtype=np.uint8)
    acc = _weights(kind, B, T + 3, r)
    n = np.array([T] * B if lens is None else lens)
    dc, da = torch.from_numpy(codes).to(DEV), torch.from_numpy(acc).to(DEV)
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    kept = torch.full((B, keep), 77, dtype=torch.int32, device=DEV)
    ws = F.Workspace()
    if in_place:
        lens_out = dl if dl is not None else torch.empty(B, dtype=torch.int32, device=DEV)
        F.cache_evict(dc, da, T, keep, recent, G=G, levels=levels, seq_lens=dl, lens_out=lens_out, kept=kept,
                      workspace=ws)
        oc, oa = dc, da
        want_c, want_a = codes.copy(), acc.copy()
    else:
        lens_out = torch.empty(B, dtype=torch.int32, device=DEV)
        Ko = (keep + 15) // 16 * 16 + 16
        want_c = r.integers(0, 256, (B, Ko, R), dtype=np.uint8)
        want_a = r.normal(size=(B, keep + 5)).astype(np.float32)
        oc, oa = torch.from_numpy(want_c).to(DEV), torch.from_numpy(want_a).to(DEV)
        F.cache_evict(dc, da, T, keep, recent, G=G, levels=levels, seq_lens=dl, out=oc, acc_out=oa, lens_out=lens_out,
                      kept=kept, workspace=ws)
        want_c, want_a = want_c.copy(), want_a.copy()
        assert np.array_equal(dc.cpu().numpy(), codes) and np.array_equal(da.cpu().numpy(), acc, equal_nan=True)
    want_k = np.full((B, keep), -1, np.int32)
    for b in range(B):
        at = O.evict(acc[b], n[b], keep, recent)
        want_c[b, :len(at)], want_a[b, :len(at)], want_k[b, :len(at)] = codes[b, at], acc[b, at], at
        if in_place:
            want_a[b, len(at):n[b]] = 0.0
            # the code bytes of freed positions are unspecified
            want_c[b, len(at):n[b]] = oc[b, len(at):n[b]].cpu().numpy()
    assert F.workspace_status(ws.buf) == F.FSQ_OK
    assert np.array_equal(lens_out.cpu().numpy(), np.minimum(n, keep))
    assert np.array_equal(kept.cpu().numpy(), want_k)
    assert np.array_equal(oa.cpu().numpy(), want_a, equal_nan=True)
    assert np.array_equal(oc.cpu().numpy(), want_c)


# rows of 128, 42, 80, 256, 144, 80, 8, 4, 3, 1 bytes: whole 16-byte pieces, and 8, 4, 2, 1
WIDTHS = [(256, 16), (84, 16), (160, 16), (256, 256), (144, 256), (320, 4), (16, 16), (8, 16), (6, 16), (4, 4), (576, 4)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("G,levels", WIDTHS)
def test_evict_widths(G, levels, in_place):
    _evict_case(3, 3001, G, levels, 1203, 100, [3001, 1500, 1203], "plain", in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signs"])
@pytest.mark.parametrize("T,keep,recent", [(1, 1, 0), (2, 1, 0), (2, 1, 1), (33, 32, 0), (1024, 1, 0), (1025, 1024, 7),
                                           (5000, 2500, 2500), (5000, 4999, 0), (5000, 6000, 10), (20000, 333, 32),
                                           (40000, 39000, 1000)])
def test_evict_weights(T, keep, recent, kind, in_place):
    lens = [T, max(0, T - 1), min(T, keep), 0, T // 2]
    _evict_case(5, T, 84, 16, keep, recent, lens, kind, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_rows(in_place):
    """More tokens than one pass of a full cluster's threads, whole rows of 16-byte pieces."""
    _evict_case(2, 150001, 256, 16, 70000, 4000, None, "ties", in_place)


def test_evict_in_place_of_many_rows_repeatedly():
    """In place, chunks of every row are moved concurrently: the same call on
    many rows, many times, always gives the oracle's rows."""
    for seed in range(8):
        _evict_case(24, 6000, 256, 16, 3000 + 100 * seed, 64, None, "plain", True, seed)


def test_evict_out_of_range_length_is_clamped_and_recorded():
    T, G = 100, 84
    codes = torch.zeros((3, 112, 42), dtype=torch.uint8, device=DEV)
    acc = torch.rand((3, T), device=DEV)
    lens = torch.tensor([50, 101, -3], dtype=torch.int32, device=DEV)
    out = torch.empty(3, dtype=torch.int32, device=DEV)
    ws = F.Workspace()
    F.cache_evict(codes, acc, T, 60, 5, G=G, seq_lens=lens, lens_out=out, workspace=ws)
    assert out.tolist() == [50, 60, 0] and F.workspace_status(ws.buf) == F.FSQ_ERR_INVALID_ARG
    F.cache_evict(codes, acc, T, 60, 5, G=G, seq_lens=out, lens_out=out, workspace=ws)
    assert out.tolist() == [50, 60, 0] and F.workspace_status(ws.buf) == F.FSQ_OK


def test_evict_captured_and_replayed():
    """Into another cache, captured; the replay sees new weights and lengths."""
    B, T, keep = 4, 2000, 700
    codes = torch.randint(0, 256, (B, T, 128), dtype=torch.uint8, device=DEV)
    acc = torch.rand((B, T), device=DEV)
    lens = torch.full((B,), T, dtype=torch.int32, device=DEV)
    out, ao = torch.zeros((B, 704, 128), dtype=torch.uint8, device=DEV), torch.zeros((B, keep), device=DEV)
    lo, kept, ws = torch.zeros_like(lens), torch.zeros((B, keep), dtype=torch.int32, device=DEV), F.Workspace()

    def call():
        F.cache_evict(codes, acc, T, keep, 50, seq_lens=lens, out=out, acc_out=ao, lens_out=lo, kept=kept, workspace=ws)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    acc.copy_(torch.rand((B, T), device=DEV))
    lens.copy_(torch.tensor([2000, 1000, 700, 3], dtype=torch.int32))
    for _ in range(2):
        g.replay()
        for b in range(B):
            at = O.evict(acc[b].cpu().numpy(), int(lens[b]), keep, 50)
            assert kept[b, :len(at)].tolist() == at.tolist() and (kept[b, len(at):] == -1).all()
            assert torch.equal(out[b, :len(at)], codes[b, torch.from_numpy(at).to(DEV)])
