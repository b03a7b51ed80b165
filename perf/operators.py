"""The operators of a state space layer, as they are measured: the scan over a prompt, the step of a single token,
the norm ahead of a projection with its 8-bit output, and the projection itself.

`run` computes them in their plain form (elementary torch operations in 32 bits), or, where `own` is true, through
the calls of gated_delta_rule_71_b200.
"""
import math

import torch

own = False

BLOCK = 128    # elements under one 8-bit scale
E4M3_MAX = 448.0
CHUNK = 128    # tokens of a chunk of the plain scan


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # the scan over a prompt batch of the headline layer's shape (B = 4, T = 4096, 2048 value channels)
        {"name": "scan batch", "op": "scan", "dtype": "bf16", "B": 4, "T": 4096, "packed": 0, "H": 32, "G": 8, "P": 64,
         "N": 128, "skip": True, "gate": True, "h0": False},
        # a packed batch that goes on from earlier states, at the decode workload's head sizes
        {"name": "scan packed", "op": "scan", "dtype": "bf16", "B": 1, "T": 32768, "packed": 8, "H": 32, "G": 16,
         "P": 128, "N": 128, "skip": True, "gate": False, "h0": True},
        # one long document: few heads in flight, so the work has to be split over its length
        {"name": "scan long", "op": "scan", "dtype": "bf16", "B": 1, "T": 131072, "packed": 0, "H": 32, "G": 1, "P": 64,
         "N": 64, "skip": True, "gate": False, "h0": False},
        # a short prompt kept in 32 bits, of no round length
        {"name": "scan exact", "op": "scan", "dtype": "fp32", "B": 1, "T": 717, "packed": 3, "H": 8, "G": 2, "P": 32,
         "N": 32, "skip": True, "gate": True, "h0": True},
        # one token of a full decode batch
        {"name": "token batch", "op": "token", "n": 256, "slots": 256, "pad": 0, "H": 32, "G": 16, "P": 128, "N": 128,
         "W": 4, "gate": True},
        # one token of a single request: latency
        {"name": "token single", "op": "token", "n": 1, "slots": 3, "pad": 0, "H": 32, "G": 8, "P": 64, "N": 128, "W": 4,
         "gate": True},
        # the norm ahead of the projection, over a prompt
        {"name": "norm prompt", "op": "norm", "dtype": "bf16", "rows": 16384, "D": 4096, "residual": True},
        # the same for one decode batch
        {"name": "norm token", "op": "norm", "dtype": "bf16", "rows": 32, "D": 2048, "residual": True},
        # a width that ends inside a block, from 32-bit activations, without a residual
        {"name": "norm ragged", "op": "norm", "dtype": "fp32", "rows": 1111, "D": 1000, "residual": False},
        # the projection of a prompt into the conv row
        {"name": "matmul prompt", "op": "matmul", "M": 4096, "N": 14336, "K": 4096, "out": "bf16"},
        # the projection of one decode batch, of no round size
        {"name": "matmul ragged", "op": "matmul", "M": 77, "N": 6176, "K": 2064, "out": "bf16"},
        # the projection of a single token: the weights' bytes
        {"name": "matmul token", "op": "matmul", "M": 1, "N": 8192, "K": 4096, "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "token", "norm", "matmul"])
    if op == "scan":
        f32 = rng.random() < 0.25
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        P, N = rng.choice([32, 64, 64, 128]), rng.choice([32, 64, 128, 128])
        packed = rng.choice([0, 0, 1, 5, 13])
        B = 1 if packed else rng.choice([1, 2, 3])
        most = min(65536, int((1 << 28) / (B * H * max(P, N))))
        T = max(packed, _log(rng, 1, min(most, 1500) if f32 else most))
        return {"op": "scan", "dtype": "fp32" if f32 else "bf16", "B": B, "T": T, "packed": packed, "H": H, "G": G,
                "P": P, "N": N, "skip": rng.random() < 0.7, "gate": rng.random() < 0.5, "h0": rng.random() < 0.5}
    if op == "token":
        G = rng.choice([1, 2, 8])
        H = G * rng.choice([1, 3, 4])
        P, N = rng.choice([32, 64, 128]), rng.choice([32, 64, 128])
        n = _log(rng, 1, min(384, (1 << 27) // (H * P * N)))
        return {"op": "token", "n": n, "slots": n + rng.randrange(9), "pad": rng.randrange(2) * (n // 3), "H": H, "G": G,
                "P": P, "N": N, "W": rng.choice([2, 3, 4]), "gate": rng.random() < 0.5}
    if op == "norm":
        D = _log(rng, 64, 16384)
        D = D if rng.random() < 0.4 else (D + 7) // 8 * 8
        return {"op": "norm", "dtype": rng.choice(["bf16", "bf16", "fp32"]), "rows": _log(rng, 1, (1 << 26) // D // 2),
                "D": D, "residual": rng.random() < 0.6}
    N, K = _log(rng, 16, 14336), 16 * _log(rng, 1, 512)
    return {"op": "matmul", "M": _log(rng, 1, min(8192, max(1, (1 << 37) // (N * K)))), "N": N, "K": K,
            "out": rng.choice(["bf16", "bf16", "fp32"])}


def work(c):
    e = 2 if c.get("dtype", "bf16") == "bf16" else 4
    if c["op"] == "scan":
        rows, H, G, P, N = c["B"] * c["T"], c["H"], c["G"], c["P"], c["N"]
        seqs = c["packed"] or c["B"]
        by = rows * e * (2 * H * P + 2 * G * N + H + (H * P if c["gate"] else 0)) + seqs * H * N * P * 4 * (2 if c["h0"] else 1)
        return {"bytes": by, "flops": rows * H * 5 * N * P}
    if c["op"] == "token":
        n, H, G, P, N, W = c["n"] - c["pad"], c["H"], c["G"], c["P"], c["N"], c["W"]
        C = H * P + 2 * G * N
        by = n * (8 * H * N * P + 2 * (C + H) + 4 * C * (W - 1) + 2 * H * P * (2 if c["gate"] else 1)) + 4 * C * (W + 1)
        return {"bytes": by, "flops": n * (H * 5 * N * P + 2 * C * W)}
    if c["op"] == "norm":
        rows, D = c["rows"], c["D"]
        by = rows * D * (e + 1 + (2 * e if c["residual"] else 0)) + rows * -(-D // BLOCK) * 4 + 4 * D
        return {"bytes": by, "flops": rows * D * 6}
    M, N, K = c["M"], c["N"], c["K"]
    kb = -(-K // BLOCK)
    return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // BLOCK)) + M * N * (2 if c["out"] == "bf16" else 4),
            "flops": 2 * M * N * K}


# ----------------------------------------------------------------------- inputs

def _lengths(c, g):
    if not c["packed"]:
        return [c["T"]] * c["B"]
    if c["packed"] == 1:
        return [c["T"]]
    cuts = torch.randint(0, c["T"] + 1, (c["packed"] - 1,), generator=g).sort().values.tolist()
    edges = [0] + cuts + [c["T"]]
    return [b - a for a, b in zip(edges, edges[1:])]


def _heads(H, rnd):
    A_log = rnd(H, uniform=True) * math.log(16.0)
    dt = torch.exp(rnd(H, uniform=True) * math.log(100.0) + math.log(1e-3))
    return A_log, torch.log(torch.expm1(dt.double())).float()


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def rnd(*shape, uniform=False):
        f = torch.rand if uniform else torch.randn
        return f(shape, generator=g, device=dev, dtype=torch.float32)

    s = {"case": c}
    if c["op"] == "scan":
        ty = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        B, T, H, G, P, N = (c[k] for k in ("B", "T", "H", "G", "P", "N"))
        # the row as the short convolution leaves it, [x | B | C]: the scan reads slices of it
        row = torch.nn.functional.silu(rnd(B, T, H * P + 2 * G * N)).to(ty)
        s["x"] = row[..., :H * P].unflatten(-1, (H, P))
        s["Bm"] = row[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["Cm"] = row[..., H * P + G * N:].unflatten(-1, (G, N))
        s["dt"] = rnd(B, T, H).to(ty)
        s["z"] = rnd(B, T, H, P).to(ty) if c["gate"] else None
        s["A_log"], s["dt_bias"] = _heads(H, rnd)
        s["D"] = 1.0 + 0.1 * rnd(H) if c["skip"] else None
        s["lengths"] = _lengths(c, torch.Generator().manual_seed(seed))
        s["h0"] = 0.1 * rnd(len(s["lengths"]), H, N, P) if c["h0"] else None
        s["cu"] = (torch.tensor([0] + torch.tensor(s["lengths"]).cumsum(0).tolist(), dtype=torch.int32, device=dev)
                   if c["packed"] else None)
    elif c["op"] == "token":
        n, H, G, P, N, W = (c[k] for k in ("n", "H", "G", "P", "N", "W"))
        C = H * P + 2 * G * N
        s["row"], s["dt"] = rnd(n, C).bfloat16(), rnd(n, H).bfloat16()
        s["z"] = rnd(n, H * P).bfloat16() if c["gate"] else None
        s["conv_w"], s["conv_bias"] = rnd(C, W) / math.sqrt(W), 0.1 * rnd(C)
        s["conv_state"] = rnd(c["slots"], C, W - 1).bfloat16()
        s["A_log"], s["dt_bias"] = _heads(H, rnd)
        s["D"] = 1.0 + 0.1 * rnd(H)
        s["state"] = 0.1 * rnd(c["slots"], H, N, P)
        idx = torch.randperm(c["slots"], generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
        idx[:c["pad"]] = -1
        s["idx"] = idx.to(dev)
    elif c["op"] == "norm":
        ty = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["x"] = rnd(c["rows"], c["D"]).to(ty)
        s["residual"] = (3.0 * rnd(c["rows"], c["D"])).to(ty) if c["residual"] else None
        s["weight"] = 1.0 + 0.1 * rnd(c["D"])
    else:
        M, N, K = c["M"], c["N"], c["K"]
        kb = -(-K // BLOCK)
        s["a"] = (100.0 * rnd(M, K)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["w"] = (100.0 * rnd(N, K)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["a_scales"] = 0.01 * torch.exp(0.3 * rnd(M, kb))
        s["w_scales"] = 0.01 / math.sqrt(K) * torch.exp(0.3 * rnd(-(-N // BLOCK), kb))
    return s


# ------------------------------------------------------------------- plain forms

def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v)))


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _chunks(lengths, dev):
    """The rows of each chunk of each sequence, -1 behind a sequence's last; and each chunk's sequence."""
    n = torch.tensor(lengths)
    per = (n + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(lengths)), per)
    first = torch.arange(len(seq)) - (per.cumsum(0) - per)[seq]
    at = first[:, None] * CHUNK + torch.arange(CHUNK)
    rows = torch.where(at < n[seq][:, None], at + (n.cumsum(0) - n)[seq][:, None], -1)
    return rows.to(dev), seq.to(dev)


def _scan(s):
    c = s["case"]
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    per = H // G
    ty = s["x"].dtype
    rows, seq = _chunks(s["lengths"], s["x"].device)
    live = rows >= 0
    at = rows.clamp(min=0)

    def cut(t):  # [B, T, ...] -> [chunks, CHUNK, ...], zeros behind the sequences
        t = t.flatten(0, 1)[at].float()
        return t.masked_fill(~live.view(*live.shape, *([1] * (t.dim() - 2))), 0.0)

    x, Bm, Cm = cut(s["x"]), cut(s["Bm"]), cut(s["Cm"])
    dt = _softplus(s["dt"].flatten(0, 1).float() + s["dt_bias"])[at] * live[..., None]
    # sums of logarithms in 64 bits: a difference of far ones is what counts
    cum = torch.cumsum(dt.double() * -torch.exp(s["A_log"].double()), 1)         # [chunks, CHUNK, H]
    total = cum[:, -1]                                                           # [chunks, H]
    xdt = x * dt[..., None]
    # within a chunk
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    cumh = cum.transpose(1, 2)
    decay = torch.exp((cumh[..., :, None] - cumh[..., None, :]).masked_fill(~low, -math.inf).float())
    pairs = Cm.transpose(1, 2) @ Bm.permute(0, 2, 3, 1)                          # [chunks, G, CHUNK, CHUNK]
    y = ((pairs.repeat_interleave(per, 1) * decay) @ xdt.transpose(1, 2)).transpose(1, 2)
    del decay, pairs
    # what each chunk adds to the state, and the state that enters each chunk
    to_end = torch.exp((total[:, None] - cum).float())
    added = Bm.repeat_interleave(per, 2).permute(0, 2, 3, 1) @ (xdt * to_end[..., None]).transpose(1, 2)
    upto = torch.cumsum(total, 0).T                                              # [H, chunks]
    before = upto - total.T
    k = torch.arange(len(seq), device=x.device)
    linked = (seq[:, None] == seq[None, :]) & (k[:, None] > k[None, :])
    pull = torch.exp((before[:, :, None] - upto[:, None, :]).masked_fill(~linked, -math.inf)).float()
    enter = (pull @ added.transpose(0, 1).flatten(2)).unflatten(2, (N, P)).transpose(0, 1)
    del pull
    starts = torch.zeros(len(s["lengths"]) + 1, dtype=torch.float64, device=x.device).repeat(H, 1)
    if s["h0"] is not None:
        head = torch.full((len(s["lengths"]),), 0, device=x.device).scatter_reduce(0, seq, k, "amin", include_self=False)
        starts = before[:, head[seq]] if len(seq) else before
        enter = enter + torch.exp(before - starts).T.float()[..., None, None] * s["h0"][seq]
    y = y + torch.exp(cum.float())[..., None] * (Cm.repeat_interleave(per, 2).transpose(1, 2) @ enter).transpose(1, 2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * x
    out = torch.zeros(c["B"] * c["T"], H, P, device=x.device)
    out[rows[live]] = y[live]
    if s["z"] is not None:
        out = out * _silu(s["z"].flatten(0, 1).float())
    # a sequence's last state: that behind its last chunk, or the one it came with
    left = torch.exp(total).float()[..., None, None] * enter + added
    hT = s["h0"].clone() if s["h0"] is not None else torch.zeros(len(s["lengths"]), H, N, P, device=x.device)
    last = torch.nn.functional.pad(seq[1:] != seq[:-1], (0, 1), value=True) if len(seq) else seq.bool()
    hT[seq[last]] = left[last]
    return {"y": out.to(ty).view(c["B"], c["T"], H, P), "hT": hT}


def _token(s):
    c = s["case"]
    n, H, G, P, N = c["n"], c["H"], c["G"], c["P"], c["N"]
    per = H // G
    live = s["idx"] >= 0
    slot = s["idx"].long().clamp(min=0)
    window = torch.cat([s["conv_state"][slot], s["row"][..., None]], -1)         # [n, C, W]
    v = _silu(s["conv_bias"] + (s["conv_w"] * window.float()).sum(-1))
    x = v[:, :H * P].view(n, H, 1, P)
    Bm = v[:, H * P:H * P + G * N].view(n, G, N, 1).repeat_interleave(per, 1)
    Cm = v[:, H * P + G * N:].view(n, G, N, 1).repeat_interleave(per, 1)
    dt = _softplus(s["dt"].float() + s["dt_bias"])[..., None, None]
    a = torch.exp(-torch.exp(s["A_log"])[:, None, None] * dt)
    h = a * s["state"][slot] + dt * Bm * x
    y = (h * Cm).sum(2) + s["D"][:, None] * x[:, :, 0]
    if s["z"] is not None:
        y = y * _silu(s["z"].float()).view(n, H, P)
    y = torch.where(live[:, None, None], y, 0.0)
    s["state"][slot[live]] = h[live]
    s["conv_state"][slot[live]] = window[live][..., 1:]
    return {"y": y.bfloat16(), "state": s["state"], "conv_state": s["conv_state"]}


def _blocks(v):
    D = v.shape[-1]
    v = torch.nn.functional.pad(v, (0, -D % BLOCK))
    return v.unflatten(-1, (-1, BLOCK))


def _norm(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
        s["residual"].copy_(v)
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    y = _blocks(y)
    most = y.abs().amax(-1, keepdim=True)
    scales = torch.where(most > 0, most / E4M3_MAX, 1.0)
    q = (y / scales).to(torch.float8_e4m3fn)
    return {"q": q.flatten(1)[:, :v.shape[-1]].contiguous(), "scales": scales[..., 0], "residual": s["residual"]}


def _matmul(s):
    c = s["case"]
    a = (_blocks(s["a"].float()) * s["a_scales"][..., None]).flatten(1)
    ws = s["w_scales"].repeat_interleave(BLOCK, 0)[:c["N"]]
    w = (_blocks(s["w"].float()) * ws[..., None]).flatten(1)
    return {"out": (a @ w.T).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)}


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"scan": _scan, "token": _token, "norm": _norm, "matmul": _matmul}[c["op"]](s)


# ------------------------------------------------------------- the framework's calls

def _own(s):
    import gated_delta_rule_71_b200 as gdn
    c = s["case"]
    if c["op"] == "scan":
        y, hT = gdn.ssm_scan(s["x"], s["dt"], s["Bm"], s["Cm"], s["A_log"], s["dt_bias"], D=s["D"], z=s["z"], h0=s["h0"],
                             cu_seqlens=s["cu"])
        return {"y": y, "hT": hT}
    if c["op"] == "token":
        y = gdn.ssm_decode_step(s["row"], s["dt"], s["conv_w"], s["conv_state"], s["A_log"], s["dt_bias"], s["state"],
                                c["H"], c["G"], c["P"], c["N"], D=s["D"], z=s["z"], conv_bias=s["conv_bias"],
                                state_indices=s["idx"])
        return {"y": y, "state": s["state"], "conv_state": s["conv_state"]}
    if c["op"] == "norm":
        q, scales = gdn.rmsnorm_fp8(s["x"], s["weight"], residual=s["residual"], eps=1e-6)
        return {"q": q, "scales": scales, "residual": s["residual"]}
    return {"out": gdn.fp8_matmul(s["a"], s["a_scales"], s["w"], s["w_scales"],
                                  out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)}


# ------------------------------------------------------- the definitions in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    sp = torch.nn.functional.softplus
    silu = torch.nn.functional.silu
    if c["op"] == "scan":
        # token by token, every sequence at its own place
        H, G, P, N = c["H"], c["G"], c["P"], c["N"]
        lens = torch.tensor(s["lengths"], device="cuda")
        first = lens.cumsum(0) - lens
        x, Bm, Cm = (d[k].flatten(0, 1) for k in ("x", "Bm", "Cm"))
        dt = sp(d["dt"].flatten(0, 1) + d["dt_bias"])
        a = torch.exp(-d["A_log"].exp() * dt)
        h = d["h0"].clone() if c["h0"] else torch.zeros(len(lens), H, N, P, dtype=torch.float64, device="cuda")
        hg = h.view(-1, G, H // G, N, P)
        y = torch.zeros(c["B"] * c["T"], H, P, dtype=torch.float64, device="cuda")
        xdt = (x * dt[..., None]).view(-1, G, H // G, 1, P)
        same = len(set(s["lengths"])) == 1
        for t in range(max(s["lengths"])):
            on = slice(None) if same else torch.nonzero(lens > t)[:, 0]
            r = first[on] + t
            new = hg[on] * a[r].view(-1, G, H // G, 1, 1) + Bm[r][:, :, None, :, None] * xdt[r]
            hg[on] = new
            y[r] = torch.matmul(Cm[r][:, :, None, None, :], new).reshape(-1, H, P)
        if c["skip"]:
            y += d["D"][:, None] * x
        if c["gate"]:
            y *= silu(d["z"].flatten(0, 1))
        return {"y": y.view(c["B"], c["T"], H, P), "hT": h}
    if c["op"] == "token":
        H, G, P, N, W = c["H"], c["G"], c["P"], c["N"], c["W"]
        y = torch.zeros(c["n"], H, P, dtype=torch.float64, device="cuda")
        for r, at in enumerate(s["idx"].tolist()):
            if at < 0:
                continue
            win = torch.cat([d["conv_state"][at], d["row"][r][:, None]], 1)
            v = silu((d["conv_w"] * win).sum(1) + d["conv_bias"])
            x, Bm, Cm = v[:H * P].view(H, P), v[H * P:H * P + G * N].view(G, N), v[H * P + G * N:].view(G, N)
            dt = sp(d["dt"][r] + d["dt_bias"])
            grp = torch.arange(H, device="cuda") // (H // G)
            h = d["state"][at] * torch.exp(-d["A_log"].exp() * dt)[:, None, None]
            h = h + torch.einsum("hn,hp,h->hnp", Bm[grp], x, dt)
            y[r] = torch.einsum("hnp,hn->hp", h, Cm[grp]) + d["D"][:, None] * x
            if c["gate"]:
                y[r] *= silu(d["z"][r].view(H, P))
            d["state"][at] = h
            d["conv_state"][at] = win[:, 1:]
        return {"y": y, "state": d["state"], "conv_state": d["conv_state"]}
    if c["op"] == "norm":
        v = d["x"] + (d["residual"] if c["residual"] else 0.0)
        y = v / (v.pow(2).sum(1, keepdim=True) / c["D"] + 1e-6).sqrt() * d["weight"]
        top = torch.stack([b.abs().amax(1) for b in y.split(BLOCK, 1)], 1)
        scales = torch.where(top > 0, top / E4M3_MAX, 1.0)
        # the values before their rounding to 8 bits: one on the border of two 8-bit numbers may become either
        q = torch.cat([b / scales[:, j:j + 1] for j, b in enumerate(y.split(BLOCK, 1))], 1)
        return {"q": q, "scales": scales, "residual": v if c["residual"] else None}
    out = 0.0
    for j, (a, w) in enumerate(zip(d["a"].split(BLOCK, 1), d["w"].split(BLOCK, 1))):
        of_row = d["w_scales"][:, j][torch.arange(c["N"], device="cuda") // BLOCK]
        out = out + (a * d["a_scales"][:, j:j + 1]) @ (w * of_row[:, None]).T
    return {"out": out}
