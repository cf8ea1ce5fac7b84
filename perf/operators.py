"""Cases of the serving operators around a bit-packed FSQ code cache, in two forms: the library's calls (`own`)
and plain torch.

  norm_rope  RMS norm of every query and key head with the rotary positions in the same pass
  prefix     decode attention of a batch whose rows share one long prefix of cached tokens
  weights    attention weight of every cached token, summed over the query heads and accumulated over steps
  evict      keep a row's recent tokens and those of the largest accumulated weight, packed into a smaller cache

Layouts are the library's: 128-wide heads; a token's row is G codes of log2(levels) bits, the first in the lowest
bits; W_kv [2 * n_kv * 128, G] holds the key rows of every kv head, then the value rows.
"""
import math

import numpy as np
import torch

own = False

D = 128
EPS = 1e-6
BASE = 1.0e6
BITS = {4: 2, 16: 4, 256: 8}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of one sequence: 32 query heads, 8 key heads
        dict(name="norm_rope_decode_1", op="norm_rope", n=1, n_q=32, n_k=8, far=40000, fused=False),
        # a chunk of an odd length in a long context, heads taken out of a fused q, k, v projection
        dict(name="norm_rope_chunk_16383", op="norm_rope", n=16383, n_q=32, n_k=8, far=1 << 20, fused=True),
        # a small model's batch on a short system prompt, a few tokens of its own per row
        dict(name="prefix_small", op="prefix", B=4, n_q=16, n_kv=8, G=256, levels=16, Tp=1024, T=16, ragged=False),
        # 8B-shaped layer at 42 B per token, a document asked 16 ragged questions
        dict(name="prefix_84_ragged", op="prefix", B=16, n_q=32, n_kv=8, G=84, levels=16, Tp=32767, T=513, ragged=True),
        # the same layer with 8-bit codes at 80 B per token, an odd batch
        dict(name="prefix_8bit_33", op="prefix", B=33, n_q=32, n_kv=8, G=80, levels=256, Tp=8192, T=200, ragged=True),
        # 8B-shaped layer at 128 B per token, the longest shared context
        dict(name="prefix_131072", op="prefix", B=16, n_q=32, n_kv=8, G=256, levels=16, Tp=131072, T=1024, ragged=True),
        # the first step of one short sequence
        dict(name="weights_1024", op="weights", B=1, n_q=16, n_kv=8, G=256, levels=16, T=1024, ragged=False, steps=0),
        # 2-bit codes at 80 B per token, a ragged batch
        dict(name="weights_2bit_ragged", op="weights", B=5, n_q=32, n_kv=8, G=320, levels=4, T=9001, ragged=True, steps=3),
        # 8B-shaped layer, the largest cache
        dict(name="weights_131072", op="weights", B=16, n_q=32, n_kv=8, G=256, levels=16, T=131072, ragged=False,
             steps=16),
        # one row brought back to its budget
        dict(name="evict_2048", op="evict", B=1, G=256, levels=16, T=2048, keep=1024, recent=128, ragged=False),
        # 42-byte rows, odd lengths, some rows still below the budget
        dict(name="evict_84_ragged", op="evict", B=8, G=84, levels=16, T=20001, keep=8191, recent=1000, ragged=True),
        # the longest prompts halved
        dict(name="evict_131072", op="evict", B=16, G=256, levels=16, T=131072, keep=65536, recent=4096, ragged=False),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "prefix", "weights", "evict"])
    if op == "norm_rope":
        return dict(op=op, n=_spread(rng, 1, 16383), n_q=rng.choice([16, 32]), n_k=rng.choice([0, 8]),
                    far=_spread(rng, 1, 1 << 20), fused=rng.random() < 0.5)
    G, levels = rng.choice([(256, 16), (84, 16), (160, 16), (80, 256), (144, 256)])
    B = _spread(rng, 1, 33)
    if op == "prefix":
        return dict(op=op, B=B, n_q=rng.choice([16, 32]), n_kv=8, G=G, levels=levels,
                    Tp=_spread(rng, 64, min(131072, (16 * 131072) // B)), T=_spread(rng, 1, 1024),
                    ragged=rng.random() < 0.5)
    T = _spread(rng, 64, min(131072, (16 * 131072) // B))
    if op == "weights":
        if rng.random() < 0.25:
            G, levels = 320, 4
            T = min(T, 60000)
        return dict(op=op, B=B, n_q=rng.choice([16, 32]), n_kv=8, G=G, levels=levels, T=T,
                    ragged=rng.random() < 0.5, steps=rng.randrange(0, 20))
    keep = max(1, int(T * rng.uniform(0.1, 0.9)))
    return dict(op=op, B=B, G=G, levels=levels, T=T, keep=keep, recent=int(keep * rng.uniform(0.0, 0.5)),
                ragged=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "norm_rope":
        e = c["n"] * (c["n_q"] + c["n_k"]) * D
        return {"bytes": 4 * e + 4 * c["n"] + 4 * D, "flops": 8 * e}
    R = c["G"] * BITS[c["levels"]] // 8
    lens = _lengths(c)
    if c["op"] == "prefix":
        small = 4 * c["B"] * c["n_q"] * D + 4 * c["n_kv"] * D * c["G"]  # q, o and W_kv
        pairs = c["B"] * c["Tp"] + sum(lens)
        return {"bytes": (c["Tp"] + sum(lens)) * R + small,
                "flops": 4 * c["n_q"] * c["G"] * pairs + 4 * c["B"] * c["n_q"] * D * c["G"]}
    if c["op"] == "weights":
        small = 2 * c["B"] * c["n_q"] * D + 2 * c["n_kv"] * D * c["G"]  # q and W_k
        return {"bytes": sum(lens) * (R + 8) + small, "flops": 2 * c["n_q"] * c["G"] * sum(lens)}
    kept = sum(min(n, c["keep"]) for n in lens)
    return {"bytes": 4 * sum(lens) + kept * (2 * R + 8), "flops": 0}


def _lengths(case):
    """Tokens of each row: all of T, or spread over 1 .. T (the longest row first)."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [max(1, T - (b * 7919 + 13 * b * b) % T) for b in range(B)]


# ---------------------------------------------------------------- inputs
def _normal(shape, std, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _codes(rows, G, levels, gen):
    """Packed codes [rows, G * bits / 8] of pre-activations N(0, 4), quantised as the append does."""
    h, delta, b = (levels - 1) / 2.0, 0.5, BITS[levels]
    out = torch.empty((rows, G * b // 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // G)
    for r in range(0, rows, step):
        u = torch.randn((min(step, rows - r), G), generator=gen, device="cuda") * 2.0
        n = (torch.round(h * torch.tanh(u + math.atanh(delta / h)) - delta) + levels // 2).to(torch.uint8)
        n = n.view(n.shape[0], -1, 8 // b)
        w = n[:, :, 0].clone()
        for k in range(1, 8 // b):
            w |= n[:, :, k] << (k * b)
        out[r:r + n.shape[0]] = w
    return out


def _cache(B, T, G, levels, gen):
    Tm = (T + 15) // 16 * 16  # the rows' stride is a multiple of 16 bytes
    return _codes(B * Tm, G, levels, gen).view(B, Tm, -1)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if c["op"] == "norm_rope":
        n, n_q, n_k = c["n"], c["n_q"], c["n_k"]
        heads = n_q + 2 * n_k if c["fused"] else n_q + n_k
        x = _normal((n, heads, D), 1.7, gen)  # projections before their norm
        c["q"], c["k"] = x[:, :n_q], x[:, n_q:n_q + n_k] if n_k else None
        if not c["fused"]:
            c["q"] = c["q"].contiguous()
            c["k"] = c["k"].contiguous() if n_k else None
        c["q_gain"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)
        c["k_gain"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)
        if n > 1024:  # a chunk: positions in a row
            c["pos"] = (torch.arange(n, device="cuda") + c["far"]).to(torch.int32)
        else:  # a decode batch: each row at its own position
            c["pos"] = torch.randint(0, c["far"] + 1, (n,), generator=gen, device="cuda").to(torch.int32)
        c["q_out"] = torch.empty((n, n_q, D), dtype=torch.bfloat16, device="cuda")
        c["k_out"] = torch.empty((n, n_k, D), dtype=torch.bfloat16, device="cuda") if n_k else None
        return c
    B, G, L, T = c["B"], c["G"], c["levels"], c["T"]
    c["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
    if c["op"] == "evict":
        c["codes"] = _cache(B, T, G, L, gen)
        # weights as steps leave them: many small ones, a few large, tokens never looked at
        a = torch.empty((B, T), device="cuda").exponential_(1.0, generator=gen).pow_(3.0)
        a[torch.rand((B, T), generator=gen, device="cuda") < 0.05] = 0.0
        c["acc"] = a
        c["out"] = torch.zeros((B, (c["keep"] + 15) // 16 * 16, c["codes"].shape[2]), dtype=torch.uint8, device="cuda")
        c["acc_out"] = torch.zeros((B, c["keep"]), device="cuda")
        c["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        c["kept"] = torch.zeros((B, c["keep"]), dtype=torch.int32, device="cuda")
        if own:
            import fsq_latent_decode_b200 as F
            c["ws"] = F.Workspace("cuda")
        return c
    n_q, n_kv = c["n_q"], c["n_kv"]
    c["W"] = _normal((2 * n_kv * D, G), math.sqrt(1.0 / G) * 16 / L, gen)
    c["q"] = _normal((B, n_q, D), 1.0, gen)
    c["codes"] = _cache(B, T, G, L, gen)
    if c["op"] == "prefix":
        c["prefix"] = _codes(c["Tp"], G, L, gen)
        c["o"] = torch.empty((B, n_q, D), dtype=torch.bfloat16, device="cuda")
    else:
        a = torch.empty((B, T), device="cuda").exponential_(1.0, generator=gen)
        c["acc"] = a * (c["steps"] * n_q / T)
    if own:
        import fsq_latent_decode_b200 as F
        c["opts"], c["ws"] = F.attn_opts(seq_lens=c["lens"], levels=L), F.Workspace("cuda")
    return c


# ---------------------------------------------------------------- one pass
def run(state):
    c = state
    if own:
        import fsq_latent_decode_b200 as F
        if c["op"] == "norm_rope":
            F.qk_norm_rope(c["q"], c["k"], c["q_gain"], c["k_gain"], positions=c["pos"], eps=EPS, rope_base=BASE,
                           q_out=c["q_out"], k_out=c["k_out"])
            return [c["q_out"], c["k_out"]] if c["n_k"] else [c["q_out"]]
        if c["op"] == "prefix":
            F.decode_attn_prefix(c["q"], c["prefix"], c["codes"], c["W"], c["Tp"], c["T"], c["n_kv"], c["G"],
                                 opts=c["opts"], workspace=c["ws"], out=c["o"])
            return [c["o"]]
        if c["op"] == "weights":
            F.attn_weights(c["q"], c["codes"], c["W"], c["acc"], c["T"], c["n_kv"], c["G"], opts=c["opts"],
                           workspace=c["ws"])
            return [c["acc"]]
        F.cache_evict(c["codes"], c["acc"], c["T"], c["keep"], c["recent"], G=c["G"], levels=c["levels"],
                      seq_lens=c["lens"], out=c["out"], acc_out=c["acc_out"], lens_out=c["lens_out"],
                      kept=c["kept"], workspace=c["ws"])
    elif c["op"] == "norm_rope":
        _plain_norm_rope(c, c["q"], c["q_gain"], c["q_out"])
        if c["n_k"]:
            _plain_norm_rope(c, c["k"], c["k_gain"], c["k_out"])
            return [c["q_out"], c["k_out"]]
        return [c["q_out"]]
    elif c["op"] == "prefix":
        return [_plain_prefix(c)]
    elif c["op"] == "weights":
        return [_plain_weights(c)]
    else:
        _plain_evict(c)
    # the codes are moved, not computed: the packed bytes themselves have to be equal
    return [c["out"], c["acc_out"], c["lens_out"], c["kept"]]


def _plain_norm_rope(c, x, gain, out):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
    inv = BASE ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    ang = c["pos"].double()[:, None] * inv  # far positions: 64 bits until the angle is taken
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = y[..., :D // 2], y[..., D // 2:]
    out.copy_(torch.cat([a * cos - b * sin, a * sin + b * cos], -1))


def _levels(codes, levels):
    """Packed codes [..., R] -> levels [..., G] in fp32."""
    b = BITS[levels]
    shift = torch.arange(0, 8, b, device=codes.device, dtype=torch.uint8)
    n = (codes.unsqueeze(-1) >> shift) & ((1 << b) - 1)
    return n.flatten(-2).float() - levels // 2


def _query(c):
    """The queries in latent coordinates, scaled: [B, n_q, G]."""
    grp = c["n_q"] // c["n_kv"]
    wk = c["W"][:c["n_kv"] * D].float().view(c["n_kv"], D, c["G"])
    q = c["q"].float().view(c["B"], c["n_kv"], grp, D) / math.sqrt(D)
    return torch.matmul(q, wk).view(c["B"], c["n_q"], c["G"])


def _past(c):
    """True at the tokens behind a row's last one: [B, T]."""
    return torch.arange(c["T"], device="cuda") >= c["lens"][:, None]


def _plain_prefix(c):
    B, n_q, n_kv, G = c["B"], c["n_q"], c["n_kv"], c["G"]
    zp, zs = _levels(c["prefix"], c["levels"]), _levels(c["codes"][:, :c["T"]], c["levels"])
    qa = _query(c)
    sp, ss = torch.matmul(qa.view(B * n_q, G), zp.T).view(B, n_q, -1), torch.matmul(qa, zs.transpose(1, 2))
    if c["lens"] is not None:
        ss.masked_fill_(_past(c)[:, None], -math.inf)
    m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    ep, es = torch.exp(sp - m), torch.exp(ss - m)
    z = torch.matmul(ep.view(B * n_q, -1), zp).view(B, n_q, G) + torch.matmul(es, zs)
    z = z / (ep.sum(-1, keepdim=True) + es.sum(-1, keepdim=True))
    wv = c["W"][n_kv * D:].float().view(n_kv, D, G)
    o = torch.matmul(z.view(B, n_kv, n_q // n_kv, G), wv.transpose(1, 2))
    return c["o"].copy_(o.reshape(B, n_q, D))


def _plain_weights(c):
    s = torch.matmul(_query(c), _levels(c["codes"][:, :c["T"]], c["levels"]).transpose(1, 2))
    if c["lens"] is not None:
        s.masked_fill_(_past(c)[:, None], -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    return c["acc"].add_((e / e.sum(-1, keepdim=True)).sum(1))


def _plain_evict(c):
    B, T, keep = c["B"], c["T"], c["keep"]
    lens = c["lens"] if c["lens"] is not None else torch.full((B,), T, device="cuda")
    t = torch.arange(T, device="cuda")
    key = torch.where(t >= lens[:, None] - c["recent"], math.inf, c["acc"])
    key = torch.where(t >= lens[:, None], -math.inf, key)
    first = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]
    new = torch.minimum(lens, torch.tensor(keep, device="cuda"))
    there = torch.arange(keep, device="cuda") < new[:, None]
    at = torch.sort(torch.where(there, first, T), dim=1).values
    src = at.clamp(max=T - 1)
    rows = torch.gather(c["codes"], 1, src[:, :, None].expand(-1, -1, c["codes"].shape[2]))
    c["out"][:, :keep] = torch.where(there[:, :, None], rows, c["out"][:, :keep])
    c["acc_out"].copy_(torch.where(there, torch.gather(c["acc"], 1, src), c["acc_out"]))
    c["lens_out"].copy_(new)
    c["kept"].copy_(torch.where(there, at, -1))


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm_rope":
        got = [_exact_norm_rope(c, c["q"], c["q_gain"])]
        return got + [_exact_norm_rope(c, c["k"], c["k_gain"])] if c["n_k"] else got
    if c["op"] == "evict":
        return _exact_evict(c)
    lens = c["lens"].tolist() if c["lens"] is not None else [c["T"]] * c["B"]
    grp = c["n_q"] // c["n_kv"]
    W = c["W"].double().view(2, c["n_kv"], D, c["G"])
    shared = _rebuilt(c, c["prefix"], W) if c["op"] == "prefix" else None
    outs = []
    for b in range(c["B"]):
        k, v = _rebuilt(c, c["codes"][b, :lens[b]], W)
        heads, total = [], torch.zeros(lens[b], dtype=torch.float64, device="cuda")
        for j in range(c["n_kv"]):
            qj = c["q"][b, j * grp:(j + 1) * grp].double()
            kj, vj = k[j], v[j]
            if shared is not None:
                kj, vj = torch.cat([shared[0][j], kj]), torch.cat([shared[1][j], vj])
            p = torch.softmax(qj @ kj.T / math.sqrt(D), -1)
            if shared is not None:
                heads.append(p @ vj)
            else:
                total += p.sum(0)
        if shared is not None:
            outs.append(torch.cat(heads))
        else:
            acc = c["acc"][b].double()
            acc[:lens[b]] += total
            outs.append(acc)
    return [torch.stack(outs)]


def _exact_norm_rope(c, x, gain):
    """Each pair (y_i, y_{i+64}) as a complex number times e^{i angle}."""
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * gain.double()
    turn = torch.exp(torch.arange(D // 2, device="cuda", dtype=torch.float64) * (-2.0 * math.log(BASE) / D))
    ang = torch.outer(c["pos"].double(), turn)
    w = torch.polar(torch.ones_like(ang), ang)[:, None]
    z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * w
    return torch.cat([z.real, z.imag], -1)


def _rebuilt(c, codes, W):
    """Keys and values of packed rows [T, R], every one rebuilt through W_kv: two [n_kv, T, 128]."""
    b = BITS[c["levels"]]
    n = torch.stack([torch.remainder(torch.div(codes.int(), 1 << s, rounding_mode="floor"), 1 << b)
                     for s in range(0, 8, b)], -1).reshape(codes.shape[0], -1)
    z = n.double() - c["levels"] / 2
    return [z @ W[0, j].T for j in range(c["n_kv"])], [z @ W[1, j].T for j in range(c["n_kv"])]


def _exact_evict(c):
    codes, acc = c["codes"].cpu().numpy(), c["acc"].cpu().numpy().astype(np.float64)
    out, acc_out = c["out"].cpu().numpy(), c["acc_out"].cpu().numpy().astype(np.float64)
    kept = np.full((c["B"], c["keep"]), -1, np.int32)
    lens = c["lens"].tolist() if c["lens"] is not None else [c["T"]] * c["B"]
    for b, n in enumerate(lens):
        at = np.arange(n)
        if n > c["keep"]:
            old = np.arange(n - c["recent"])
            best = old[np.lexsort((old, -acc[b, old]))][:c["keep"] - c["recent"]]
            at = np.concatenate([np.sort(best), np.arange(n - c["recent"], n)])
        out[b, :len(at)], acc_out[b, :len(at)], kept[b, :len(at)] = codes[b, at], acc[b, at], at
    return [out, acc_out, np.array([min(n, c["keep"]) for n in lens], np.int32), kept]
