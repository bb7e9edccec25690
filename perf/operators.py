"""Cases for the 8-bit K/V cache and the shared-prefix attention: what a denoising loop calls per layer.

Four operators, each in a plain form (torch products, sums and exponentials in 32 bits) and as
the library's call:
  write   kv_scatter_quant          the recompute rows' fresh K/V into an e4m3 cache, one power-of-two
                                    exponent per (position, KV head) row
  read    kv_gather_quant           rows of that cache back as bf16
  attn    partial_attention_quant   attention of the recompute rows against the 8-bit cache
  prefix  prefix_attention          attention of a batch against one prefix shared by every
                                    sequence and each sequence's own cache (bf16 or 8-bit)

Shapes are the repository's workloads (8 x 64 at L 256; 32 x 128 at L 1024, 4096 and 32768;
28 query / 4 KV heads x 128 at L 2048) and sizes around them. R rows per sequence (95 = one block
of 31 masked positions and 64 recently decoded ones), ragged over a batch.
"""
from __future__ import annotations

import math

import torch

own = False

E_MIN = -110  # smallest row exponent (a row of zeros has it)


# ---------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one partial step's cache refresh at the tiny workload: a few rows, all latency
        dict(name="write_tiny", op="write", B=1, L=256, Hkv=8, D=64, R=47),
        # the partial refresh of a batch of grouped-query sequences, ragged recompute sets
        dict(name="write_gqa_batch", op="write", B=8, L=2048, Hkv=4, D=128, R=95),
        # a full step of the long context: every row is refreshed
        dict(name="write_long_full", op="write", B=1, L=32768, Hkv=32, D=128, R=32768),
        # reading the recompute rows of a batch back (inspection, migration to a bf16 cache)
        dict(name="read_gqa_batch", op="read", B=8, L=2048, Hkv=4, D=128, R=95),
        # reading a whole cache back
        dict(name="read_llada_full", op="read", B=4, L=4096, Hkv=32, D=128, R=4096),
        # one row against an odd-length cache: the single-token form
        dict(name="attn_token", op="attn", B=1, L=2047, Hq=28, Hkv=4, D=128, R=1, ragged=False),
        # the partial step of the 32-head layer, the library's headline shape
        dict(name="attn_llada", op="attn", B=1, L=1024, Hq=32, Hkv=32, D=128, R=95, ragged=False),
        # a padded batch: each sequence has its own length and recompute-set size
        dict(name="attn_gqa_batch", op="attn", B=8, L=2048, Hq=28, Hkv=4, D=128, R=95, ragged=True),
        # the long context, where the cache's bytes are the whole cost
        dict(name="attn_long", op="attn", B=1, L=32768, Hq=32, Hkv=32, D=128, R=95, ragged=False),
        # many sequences, one row each, behind one prompt of 1792 positions
        dict(name="prefix_tokens", op="prefix", B=32, Lp=1792, L=256, Hq=28, Hkv=4, D=128, R=1, ragged=False, quant=False),
        # a batch of block-wise decoders behind one few-shot prompt
        dict(name="prefix_batch", op="prefix", B=8, Lp=3840, L=256, Hq=32, Hkv=32, D=128, R=32, ragged=True, quant=False),
        # a long shared document held in 8 bits
        dict(name="prefix_long_quant", op="prefix", B=16, Lp=32512, L=256, Hq=28, Hkv=4, D=128, R=31, ragged=True, quant=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "prefix"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    if op in ("write", "read"):
        B, L = _log(rng, 1, 16), _log(rng, 2, 32768)
        while B * L * Hkv * D > 32768 * 32 * 128:
            B = max(1, B // 2)
        return dict(op=op, B=B, L=L, Hkv=Hkv, D=D, R=min(L, _log(rng, 1, max(2, L))))
    g = rng.choice([1, 2, 3, 7, 8])
    B = _log(rng, 1, 32)
    R = _log(rng, 1, 257)
    if op == "attn":
        L = max(R, _log(rng, 16, 32768))
        while B * L * Hkv * D > 32768 * 32 * 128 or B * R * Hkv * g * L > 95 * 32 * 32768:
            B, L, R = max(1, B // 2), max(R, (2 * L) // 3), max(1, (2 * R) // 3)
        return dict(op=op, B=B, L=L, Hq=g * Hkv, Hkv=Hkv, D=D, R=R, ragged=rng.random() < 0.5)
    Lp, L = _log(rng, 1, 32512), _log(rng, 1, 1024)
    R = min(R, L)
    while B * R * Hkv * g * (Lp + L) > 16 * 31 * 28 * 32768:
        B, Lp, R = max(1, B // 2), max(1, (2 * Lp) // 3), max(1, (2 * R) // 3)
    return dict(op=op, B=B, Lp=Lp, L=L, Hq=g * Hkv, Hkv=Hkv, D=D, R=R, ragged=rng.random() < 0.5, quant=rng.random() < 0.5)


def _sizes(c):
    """Recompute rows and keys of each sequence. A ragged batch spreads both downwards."""
    B, R, L = c["B"], c["R"], c["L"]
    if c["op"] in ("write", "read"):
        return [max(1, R - b * R // (2 * B)) for b in range(B)], [L] * B
    if not c["ragged"]:
        return [R] * B, [L] * B
    return [max(1, R - b * R // (2 * B)) for b in range(B)], [L - b * L // (2 * B) for b in range(B)]


def work(case):
    rows, lens = _sizes(case)
    Hkv, D = case["Hkv"], case["D"]
    n = sum(rows)
    if case["op"] in ("write", "read"):  # K and V: a bf16 row, an e4m3 row and its exponent byte
        return {"bytes": 2 * n * Hkv * (3 * D + 1) + 4 * n, "flops": 0}
    q8 = case["op"] == "attn" or case["quant"]
    Lp = case.get("Lp", 0)
    row = D + 1 if q8 else 2 * D
    keys = Lp + sum(lens)
    io = 2 * n * case["Hq"] * D * 2
    return {"bytes": 2 * keys * Hkv * row + io, "flops": 4 * case["Hq"] * D * sum(r * (Lp + s) for r, s in zip(rows, lens))}


# --------------------------------------------------------------------------------------- inputs


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, B, L, Hkv, D, spread):
    """K or V rows: normal values whose magnitude differs from position to position."""
    x = _randn(g, B, L, Hkv, D)
    x *= torch.exp2(spread * _randn(g, B, L, Hkv, 1))
    return x.to(torch.bfloat16)


def _codes(g, B, L, Hkv, D):
    """An 8-bit cache's contents: e4m3 codes of normal rows and their exponents (a cache that an earlier step wrote)."""
    x = _randn(g, B, L, Hkv, D) * 100.0
    code = x.clamp_(-448, 448).to(torch.float8_e4m3fn)
    Ls = -(-L // 16) * 16
    e = torch.randint(119, 122, (B, Hkv, Ls), generator=g, device="cuda", dtype=torch.int32)
    return code, e.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    B, L, Hkv, D = c["B"], c["L"], c["Hkv"], c["D"]
    rows, lens = _sizes(c)
    Rm = max(rows)
    s = {"case": c, "Rm": Rm, "R": torch.tensor(rows, dtype=torch.int32, device="cuda")}
    live = torch.arange(Rm, device="cuda")[None, :] < s["R"][:, None]
    if c["op"] in ("write", "read"):
        order = torch.rand(B, L, generator=g, device="cuda").argsort(1)
        idx = torch.where(live, order[:, :Rm], L).sort(1).values  # ascending positions, then padding
        s["idx"] = torch.zeros(B, L, dtype=torch.int32, device="cuda")
        s["idx"][:, :Rm] = torch.where(live, idx, 0).to(torch.int32)
        b, r = torch.nonzero(live, as_tuple=True)
        s["b"], s["r"], s["pos"] = b, r, idx[b, r]  # the plan of the plain form
        s["k8"], s["ke"] = _codes(g, B, L, Hkv, D)
        s["v8"], s["ve"] = _codes(g, B, L, Hkv, D)
        if c["op"] == "write":  # fresh rows in recompute order
            s["k"], s["v"] = (_rows(g, B, L, Hkv, D, 1.0) for _ in range(2))
        else:
            s["k"], s["v"] = (torch.zeros(B, L, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    s["q"] = _randn(g, B, L, c["Hq"], D).to(torch.bfloat16)
    s["out"] = torch.zeros(B, L, c["Hq"], D, dtype=torch.bfloat16, device="cuda")
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if c["ragged"] else None
    s["live"] = live
    if c["op"] == "attn" or c["quant"]:
        s["k8"], s["ke"] = _codes(g, B, L, Hkv, D)
        s["v8"], s["ve"] = _codes(g, B, L, Hkv, D)
        if c["op"] == "prefix":
            s["pk8"], s["pke"] = _codes(g, 1, c["Lp"], Hkv, D)
            s["pv8"], s["pve"] = _codes(g, 1, c["Lp"], Hkv, D)
    else:
        s["k"], s["v"] = (_rows(g, B, L, Hkv, D, 0.3) for _ in range(2))
        s["pk"], s["pv"] = (_rows(g, 1, c["Lp"], Hkv, D, 0.3)[0] for _ in range(2))
    return s


# --------------------------------------------------------------------------------- plain forms


def _quantise(x):
    """Codes and exponent bytes of rows x [n, Hkv, D]: the power of two that puts the row's largest value into (224, 448]."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m == 0, E_MIN, e).clamp_min(E_MIN)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _widen(code, ebyte):
    """The values that codes [B, L, Hkv, D] with exponent bytes [B, Hkv, Ls] stand for."""
    e = ebyte[:, :, : code.shape[1]].permute(0, 2, 1).to(torch.int32) - 127
    return torch.ldexp(code.float(), e[..., None])


def _plain_write(s):
    b, r, pos = s["b"], s["r"], s["pos"]
    for x, code, ebyte in ((s["k"], s["k8"], s["ke"]), (s["v"], s["v8"], s["ve"])):
        y, e = _quantise(x[b, r])
        code.view(torch.uint8)[b, pos] = y.view(torch.uint8)
        ebyte[b, :, pos] = e
    return _written(s)


def _written(s):
    L = s["case"]["L"]
    return {"k": s["k8"], "v": s["v8"], "ke": s["ke"][:, :, :L], "ve": s["ve"][:, :, :L]}


def _plain_read(s):
    b, r, pos = s["b"], s["r"], s["pos"]
    for x, code, ebyte in ((s["k"], s["k8"], s["ke"]), (s["v"], s["v8"], s["ve"])):
        e = ebyte[b, :, pos].to(torch.int32) - 127
        x[b, r] = torch.ldexp(code.view(torch.uint8)[b, pos].view(torch.float8_e4m3fn).float(), e[..., None]).to(torch.bfloat16)
    return s["k"][:, : s["Rm"]], s["v"][:, : s["Rm"]]


def _attend(q, live, k, v, n_keys, pk, pv, dtype):
    """q [B, R, Hq, D] against own keys k, v [B, L, Hkv, D] (the first n_keys[b]) and shared keys pk, pv [Lp, Hkv, D] or None."""
    B, R, Hq, D = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    g = Hq // Hkv
    q = q.to(dtype).view(B, R, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * R, D) * (1.0 / math.sqrt(D))
    sc = q @ k.to(dtype).permute(0, 2, 3, 1)
    vv = v.to(dtype).permute(0, 2, 1, 3)
    if n_keys is not None:
        dead = torch.arange(L, device=q.device) >= n_keys[:, None]
        sc = sc.masked_fill(dead[:, None, None, :], -math.inf)
        vv = vv.masked_fill(dead[:, None, :, None], 0.0)
    m = sc.amax(-1, keepdim=True)
    if pk is not None:
        qs = q.permute(1, 0, 2, 3).reshape(Hkv, B * g * R, D)
        ps = qs @ pk.to(dtype).permute(1, 2, 0)  # the shared keys once for every row of the batch
        m = torch.maximum(m, ps.amax(-1).view(Hkv, B, g * R).permute(1, 0, 2)[..., None])
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(sc - m)
    l = w.sum(-1, keepdim=True)
    o = w @ vv
    if pk is not None:
        pw = torch.exp(ps - m.permute(1, 0, 2, 3).reshape(Hkv, B * g * R, 1))
        po = pw @ pv.to(dtype).permute(1, 0, 2)
        o = o + po.view(Hkv, B, g * R, D).permute(1, 0, 2, 3)
        l = l + pw.sum(-1).view(Hkv, B, g * R).permute(1, 0, 2)[..., None]
    o = o / torch.where(l == 0, 1.0, l)
    o = o.view(B, Hkv, g, R, D).permute(0, 3, 1, 2, 4).reshape(B, R, Hq, D)
    return torch.where(live[:, :, None, None], o, 0.0)


def _plain_attention(s, dtype=torch.float32):
    c, Rm = s["case"], s["Rm"]
    pk = pv = None
    if c["op"] == "attn" or c["quant"]:
        k, v = _widen(s["k8"], s["ke"]), _widen(s["v8"], s["ve"])
        if c["op"] == "prefix":
            pk, pv = _widen(s["pk8"], s["pke"])[0], _widen(s["pv8"], s["pve"])[0]
    else:
        k, v, pk, pv = s["k"], s["v"], s["pk"], s["pv"]
    return _attend(s["q"][:, :Rm], s["live"], k, v, s["len"], pk, pv, dtype)


# ------------------------------------------------------------------------------ the library's calls


def _handle(s):
    """What a user's program makes once per layer: the shape, the caches and the scratch space."""
    import entropy_gated_kv_gb300 as E

    c = s["case"]
    p = E.Params(B=c["B"], L=c["L"], Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], D=c["D"], V=8, C_max=1, k=1)
    h = {"E": E, "p": p, "cache": E.QuantCache(s["k8"], s["v8"], s["ke"], s["ve"]) if "k8" in s else (s["k"], s["v"])}
    if c["op"] == "attn":
        h["ws"] = E.workspace(E.partial_attention_quant_workspace_size(p))
    if c["op"] == "prefix":
        h["ws"] = E.workspace(E.prefix_attention_workspace_size(p))
        h["prefix"] = E.QuantCache(s["pk8"], s["pv8"], s["pke"], s["pve"]) if c["quant"] else (s["pk"], s["pv"])
    return h


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    h, op = s["handle"], s["case"]["op"]
    E, p = h["E"], h["p"]
    if op == "write":
        E.kv_scatter_quant(p, h["cache"], s["k"], s["v"], s["idx"], s["R"])
        return _written(s)
    if op == "read":
        E.kv_gather_quant(p, h["cache"], s["idx"], s["R"], out=(s["k"], s["v"]))
        return s["k"][:, : s["Rm"]], s["v"][:, : s["Rm"]]
    if op == "attn":
        E.partial_attention_quant(p, s["q"], h["cache"], s["R"], s["out"], kv_len=s["len"], ws=h["ws"])
    else:
        E.prefix_attention(p, s["q"], h["prefix"], h["cache"], s["R"], s["out"], kv_len=s["len"], ws=h["ws"])
    return s["out"][:, : s["Rm"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "write":
        return _plain_write(state)
    if op == "read":
        return _plain_read(state)
    return _plain_attention(state).to(torch.bfloat16)


# ----------------------------------------------------------------------------------- 64 bits


def _exact_exponent(x):
    """floor(log2(amax / 448)) rounded up to the power of two that holds the row, from the logarithm, then put right by comparison."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a / 448.0)).nan_to_num(neginf=float(E_MIN)).clamp_min(E_MIN)
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)
    return torch.where((a <= 448.0 * torch.exp2(e - 1)) & (e > E_MIN), e - 1, e)


def _scale64(ebyte, L):
    return torch.exp2(ebyte[:, :, :L].double() - 127.0).transpose(1, 2).unsqueeze(-1)


def _sequence64(q, keys, values):
    """softmax(q k^T / sqrt(D)) v of one sequence: q [R, Hq, D], keys and values [n, Hkv, D], head by head."""
    R, Hq, D = q.shape
    g = Hq // keys.shape[1]
    o = torch.zeros(R, Hq, D, dtype=torch.float64, device=q.device)
    for h in range(Hq):
        z = torch.mm(q[:, h].double(), keys[:, h // g].double().T) / math.sqrt(D)
        o[:, h] = torch.mm(torch.softmax(z, 1), values[:, h // g].double())
    return o


def exact(case, seed):
    s = prepare(case, seed)
    L, Rm = case["L"], s["Rm"]
    rows, lens = _sizes(case)
    if case["op"] == "write":
        got = {}
        for n, x, code, ebyte in (("k", s["k"], s["k8"], s["ke"]), ("v", s["v"], s["v8"], s["ve"])):
            y, eb = code.double(), ebyte[:, :, :L].clone()
            for b, n_rows in enumerate(rows):
                pos = s["idx"][b, :n_rows].long()
                fresh = x[b, :n_rows].double()
                e = _exact_exponent(fresh)
                y[b, pos] = fresh * torch.exp2(-e)[..., None]
                eb[b, :, pos] = (e + 127).to(torch.uint8).T
            got[n], got[n + "e"] = y, eb
        return got
    if case["op"] == "read":
        back = []
        for code, ebyte in ((s["k8"], s["ke"]), (s["v8"], s["ve"])):
            val = code.double() * _scale64(ebyte, L)
            y = torch.zeros(case["B"], Rm, case["Hkv"], case["D"], dtype=torch.float64, device="cuda")
            for b, n_rows in enumerate(rows):
                y[b, :n_rows] = val[b, s["idx"][b, :n_rows].long()]
            back.append(y)
        return tuple(back)
    out = torch.zeros(case["B"], Rm, case["Hq"], case["D"], dtype=torch.float64, device="cuda")
    for b, (n_rows, n_keys) in enumerate(zip(rows, lens)):
        parts = []
        for n in ("k", "v"):
            if n + "8" in s:
                y = s[n + "8"][b : b + 1, :n_keys].double() * _scale64(s[n + "e"][b : b + 1], n_keys)
                y = [y[0]]
                if case["op"] == "prefix":
                    y.insert(0, (s["p" + n + "8"].double() * _scale64(s["p" + n + "e"], case["Lp"]))[0])
            else:
                y = [s["p" + n].double(), s[n][b, :n_keys].double()]
            parts.append(torch.cat(y))
        out[b, :n_rows] = _sequence64(s["q"][b, :n_rows], *parts)
    return out
