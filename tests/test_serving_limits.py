"""The serving operators at the ends of what their documentation allows, on the
GPU against 64-bit references."""
import math

import numpy as np
import pytest
import torch

import fsq_latent_decode_b200 as F
from oracle import fsq_oracle as O

from cases import decoder_weights

pytestmark = pytest.mark.gpu

DEV = "cuda"
LOG2E = math.log2(math.e)


def _dev(a):
    return (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(DEV)


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
