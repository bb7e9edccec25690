"""Cases for the paged K/V cache: what a denoising loop over a pool of pages calls per layer.

Three operators, each in a plain form (torch products, sums and exponentials in 32 bits) and as
the library's call:
  append  kv_append_paged         fresh, unrotated rows: K rotated at its position and V into the
                                  pages of a sequence, the queries rotated into an array of their own
  attn    paged_attention         the rows of a step against every key that the pages hold (one row
                                  per sequence: the single-token form)
  window  paged_window_attention  the same, with the keys near a row's position and the first few

Shapes are the repository's workloads (8 x 64; 32 x 128; 28 query / 4 KV heads x 128; L 256 to
32768) and sizes around them: R rows per sequence (95 = one block of 31 masked positions and 64
recently decoded ones; R = L is a full step), ragged over a batch, pages in no order.
"""
from __future__ import annotations

import math

import torch

own = False

THETA = 500000.0


# ---------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one new token of each sequence of a batch: all latency
        dict(name="append_tokens", op="append", B=32, L=2048, Hq=28, Hkv=4, D=128, R=1, page=16, ragged=True),
        # the partial step of a batch of grouped-query sequences, ragged recompute sets
        dict(name="append_block", op="append", B=8, L=2047, Hq=28, Hkv=4, D=128, R=95, page=32, ragged=True),
        # the first forward of a batch: every position of every prompt
        dict(name="append_full", op="append", B=4, L=4096, Hq=32, Hkv=32, D=128, R=4096, page=64, ragged=False),
        # a single token against an odd-length cache
        dict(name="attn_token", op="attn", B=1, L=2047, Hq=28, Hkv=4, D=128, R=1, page=64, ragged=False),
        # a batch of single tokens, each sequence of its own length, small pages: the cache's bytes are the cost
        dict(name="attn_tokens_batch", op="attn", B=64, L=8192, Hq=28, Hkv=4, D=128, R=1, page=16, ragged=True),
        # the partial step of the 32-head layer, the library's headline shape
        dict(name="attn_llada", op="attn", B=1, L=1024, Hq=32, Hkv=32, D=128, R=95, page=64, ragged=False),
        # a padded batch of partial steps: lengths and recompute sets of their own
        dict(name="attn_block_batch", op="attn", B=8, L=2048, Hq=28, Hkv=4, D=128, R=95, page=32, ragged=True),
        # a partial step in a long context
        dict(name="attn_long", op="attn", B=1, L=32768, Hq=32, Hkv=32, D=128, R=95, page=128, ragged=False),
        # a full step: every position against every key
        dict(name="attn_full", op="attn", B=4, L=2048, Hq=28, Hkv=4, D=128, R=2048, page=64, ragged=False),
        # a batch of single tokens far into their sequences, the last 1024 keys and four first ones
        dict(name="window_tokens", op="window", B=16, L=32767, Hq=28, Hkv=4, D=128, R=1, page=16, ragged=True, left=1023, right=0, sinks=4),
        # partial steps that see 256 positions to either side and the first 64
        dict(name="window_block", op="window", B=8, L=4096, Hq=32, Hkv=32, D=128, R=95, page=64, ragged=True, left=256, right=256, sinks=64),
        # a full step over a long document, a window to either side
        dict(name="window_full", op="window", B=1, L=16384, Hq=28, Hkv=4, D=128, R=16384, page=128, ragged=False, left=1024, right=1024, sinks=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "window"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 32])
    g = rng.choice([1, 2, 3, 7, 8])
    c = dict(op=op, B=_log(rng, 1, 64), L=_log(rng, 16, 32768), Hq=g * Hkv, Hkv=Hkv, D=D, R=1 if rng.random() < 0.3 else _log(rng, 1, 2048),
             page=rng.choice([16, 32, 64, 128, 256]), ragged=rng.random() < 0.5)
    c["R"] = min(c["R"], c["L"])
    if op == "window":
        c.update(left=rng.choice([0, 64, 255, 1024, 4096, -1]), right=rng.choice([0, 0, 64, 256, 1024]), sinks=rng.choice([0, 4, 64, 200]))
    while True:
        w = work(c)
        cells = c["B"] * c["L"] * Hkv * D  # the pool, and for the rows q, k and v
        rows = c["B"] * c["R"] * (c["Hq"] + 2 * Hkv) * D
        if w["bytes"] <= 8e8 and w["flops"] <= 4.8e11 and cells <= 32768 * 32 * 128 and rows <= 4 * 4096 * 96 * 128:
            return c
        if c["B"] > 1:
            c["B"] //= 2
        elif c["R"] > 64:
            c["R"] //= 2
        else:
            c["L"] = max(c["R"], 2 * c["L"] // 3)


def _sizes(c):
    """Rows and keys of each sequence. A ragged batch spreads both downwards."""
    B, R, L = c["B"], c["R"], c["L"]
    if not c["ragged"]:
        return [R] * B, [L] * B
    lens = [L - b * L // (2 * B) for b in range(B)]
    return [min(n, max(1, R - b * R // (2 * B))) for b, n in enumerate(lens)], lens


def _band(c, pos_lo, pos_hi, n):
    """The keys that rows at pos_lo .. pos_hi see between them: (sinks, first, end)."""
    if c["op"] != "window":
        return 0, 0, n
    lo = 0 if c["left"] < 0 else min(n, max(0, pos_lo - c["left"]))
    hi = n if c["right"] < 0 else min(n, pos_hi + c["right"] + 1)
    s = min(c["sinks"], n)
    return min(s, lo), lo, max(lo, hi)


def work(case):
    rows, lens = _sizes(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    n = sum(rows)
    if case["op"] == "append":  # q, k, v in and out, a row of each table per position, index and page
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * D * 2 + n * (4 * D + 8), "flops": 3 * n * (Hq + Hkv) * D}
    keys = cells = 0
    for r, s in zip(rows, lens):
        if case["op"] == "attn":
            keys, cells = keys + s, cells + r * s
            continue
        span = s if r == s else min(s, 4 * r)  # where the rows' positions lie (see prepare)
        near, a, e = _band(case, s - span, s - 1, s)
        keys += near + e - a
        step = max(1, r // 64)
        some = 0
        for i in range(0, r, step):
            p = s - span + (i * span) // r
            near, a, e = _band(case, p, p, s)
            some += (near + e - a) * min(step, r - i)
        cells += some
    return {"bytes": 2 * keys * Hkv * D * 2 + 2 * n * Hq * D * 2, "flops": 4 * Hq * D * cells}


# --------------------------------------------------------------------------------------- inputs


def _positions(g, r, n):
    """The recompute positions of one sequence, ascending: the last one, all, or a scattered set near the end."""
    if r == 1:
        return torch.tensor([n - 1], device="cuda")
    if r == n:
        return torch.arange(n, device="cuda")
    span = min(n, 4 * r)
    pick = torch.rand(span, generator=g, device="cuda").argsort()[:r]
    return (n - span + pick).sort().values


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    B, L, Hq, Hkv, D, page = c["B"], c["L"], c["Hq"], c["Hkv"], c["D"], c["page"]
    rows, lens = _sizes(c)
    Rm = max(rows)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)

    # the pool: as many pages as the sequences need and a few more, handed out in no order
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.rand(n_pages, generator=g, device="cuda").argsort().to(torch.int32)
    table = torch.full((B, -(-L // page)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at : at + m]
        at += m
    s = {"case": c, "Rm": Rm, "table": table, "k": randn(n_pages, page, Hkv, D), "v": randn(n_pages, page, Hkv, D)}
    s["R"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pos = [_positions(g, r, n) for r, n in zip(rows, lens)]
    s["idx"] = torch.zeros(B, Rm, dtype=torch.int32, device="cuda")
    for b, x in enumerate(pos):
        s["idx"][b, : rows[b]] = x.to(torch.int32)
    s["live"] = torch.arange(Rm, device="cuda")[None, :] < s["R"][:, None]
    if c["op"] == "append":
        s["qkv"] = randn(B, Rm, Hq + 2 * Hkv, D)  # the fused projection's output
        s["q_out"] = torch.zeros(B, Rm, Hq, D, dtype=torch.bfloat16, device="cuda")
        ang = torch.arange(L, device="cuda", dtype=torch.float64)[:, None] * THETA ** (
            -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        b, r = torch.nonzero(s["live"], as_tuple=True)
        p = s["idx"][b, r].long()
        s["b"], s["r"], s["pos"], s["slot"] = b, r, p, table[b, p // page].long() * page + p % page  # the plain form's plan
        return s
    s["q"] = randn(B, Rm, Hq, D)
    s["out"] = torch.zeros(B, Rm, Hq, D, dtype=torch.bfloat16, device="cuda")
    # the plain form's plan: for some rows at a time the slots of the keys that they see between them, and which row sees which
    step = Rm if c["op"] == "attn" and Rm <= 512 else 512
    s["plan"] = []
    host = [x.tolist() for x in pos]
    for r0 in range(0, Rm, step):
        r1 = min(Rm, r0 + step)
        keys = []
        for b in range(B):
            mine = host[b][r0:r1]
            near, a, e = _band(c, mine[0], mine[-1], lens[b]) if mine else (0, 0, 0)
            keys.append(torch.cat([torch.arange(near, device="cuda"), torch.arange(a, e, device="cuda")]))
        W = max(1, max(k.numel() for k in keys))
        j = torch.full((B, W), -1, device="cuda")
        for b, k in enumerate(keys):
            j[b, : k.numel()] = k
        slot = torch.where(j >= 0, table.long().gather(1, j.clamp_min(0) // page) * page + j.clamp_min(0) % page, 0)
        if c["op"] == "attn":
            see = (j >= 0)[:, None, :]
        else:
            p = s["idx"][:, r0:r1, None].long()
            see = (j[:, None, :] >= p - c["left"]) if c["left"] >= 0 else torch.ones_like(p, dtype=torch.bool)
            if c["right"] >= 0:
                see = see & (j[:, None, :] <= p + c["right"])
            see = (see | (j[:, None, :] < c["sinks"])) & (j >= 0)[:, None, :] & s["live"][:, r0:r1, None]
        s["plan"].append((r0, r1, slot, see))
    return s


# --------------------------------------------------------------------------------- plain forms


def _rotate(x, cs, sn):
    """x [n, H, D] turned by the angles of its positions (rotate-half), in 32 bits."""
    a, b = x.float().chunk(2, -1)
    cs, sn = cs[:, None, :], sn[:, None, :]
    return torch.cat([a * cs - b * sn, b * cs + a * sn], -1).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    b, r = s["b"], s["r"]
    x = s["qkv"][b, r]
    cs, sn = s["cos"][s["pos"]], s["sin"][s["pos"]]
    s["k"].view(-1, Hkv, D)[s["slot"]] = _rotate(x[:, Hq : Hq + Hkv], cs, sn)
    s["v"].view(-1, Hkv, D)[s["slot"]] = x[:, Hq + Hkv :]
    s["q_out"][b, r] = _rotate(x[:, :Hq], cs, sn)
    return {"k": s["k"], "v": s["v"], "q": s["q_out"]}


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv
    k, v = s["k"].view(-1, Hkv, D), s["v"].view(-1, Hkv, D)
    for r0, r1, slot, see in s["plan"]:
        n, W = r1 - r0, slot.shape[1]
        q = s["q"][:, r0:r1].float().view(B, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, D)
        sc = q @ k[slot].float().permute(0, 2, 3, 1) * (1.0 / math.sqrt(D))
        sc = sc.view(B, Hkv, g, n, W).masked_fill(~see[:, None, None], -math.inf)
        m = sc.amax(-1, keepdim=True)
        w = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
        l = w.sum(-1, keepdim=True)
        o = (w.view(B, Hkv, g * n, W) @ v[slot].float().permute(0, 2, 1, 3)).view(B, Hkv, g, n, D)
        o = (o / torch.where(l == 0, 1.0, l)).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
        s["out"][:, r0:r1] = torch.where(s["live"][:, r0:r1, None, None], o, 0.0).to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------------------ the library's calls


def _handle(s):
    """What a user's program makes once: the shape, the cache over its pool and table, the scratch space."""
    import entropy_gated_kv_gb300 as E

    c = s["case"]
    p = E.Params(B=c["B"], L=c["L"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], V=8, C_max=1, k=1)
    h = {"E": E, "p": p, "cache": E.PagedCache(s["k"], s["v"], s["table"])}
    if c["op"] == "append":
        x, Hq, Hkv = s["qkv"], c["Hq"], c["Hkv"]
        h["q"], h["k"], h["v"] = x[:, :, :Hq], x[:, :, Hq : Hq + Hkv], x[:, :, Hq + Hkv :]
    else:
        h["ws"] = E.workspace(E.paged_attention_workspace_size(p, s["Rm"]))
    return h


def _own(s):
    if "handle" not in s:
        s["handle"] = _handle(s)
    h, c = s["handle"], s["case"]
    E, p = h["E"], h["p"]
    if c["op"] == "append":
        E.kv_append_paged(p, h["cache"], h["k"], h["v"], s["R"], idx=s["idx"], rope=(s["cos"], s["sin"]), q_new=h["q"], q_out=s["q_out"])
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    if c["op"] == "attn":
        return E.paged_attention(p, s["q"], h["cache"], s["R"], s["out"], kv_len=s["len"], ws=h["ws"])
    return E.paged_window_attention(p, s["q"], h["cache"], s["R"], s["out"], left=c["left"], right=c["right"], sinks=c["sinks"],
                                    idx=s["idx"], kv_len=s["len"], ws=h["ws"])


def run(state):
    if own:
        return _own(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


# ----------------------------------------------------------------------------------- 64 bits


def _turn64(x, cs, sn):
    """Pairs (i, i + D/2) of x [n, H, D] as complex numbers times cos + i sin."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h].double(), x[..., h:].double()) * torch.complex(cs.double(), sn.double())[:, None, :]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    rows, lens = _sizes(case)
    if case["op"] == "append":
        k, v, q = s["k"].double(), s["v"].double(), s["q_out"].double()
        for b, n in enumerate(rows):
            pos = s["idx"][b, :n].long()
            x, cs, sn = s["qkv"][b, :n], s["cos"][pos], s["sin"][pos]
            where = (s["table"][b].long()[pos // page], pos % page)
            k[where] = _turn64(x[:, Hq : Hq + Hkv], cs, sn)
            v[where] = x[:, Hq + Hkv :].double()
            q[b, :n] = _turn64(x[:, :Hq], cs, sn)
        return {"k": k, "v": v, "q": q}
    g = Hq // Hkv
    out = torch.zeros(case["B"], s["Rm"], Hq, D, dtype=torch.float64, device="cuda")
    for b, (r, n) in enumerate(zip(rows, lens)):
        pages = s["table"][b, : -(-n // page)].long()
        keys, values = (s[x][pages].reshape(-1, Hkv, D)[:n] for x in ("k", "v"))
        for r0 in range(0, r, 1024):
            r1 = min(r, r0 + 1024)
            pos = s["idx"][b, r0:r1].long()
            a, e = 0, n
            if case["op"] == "window" and case["sinks"] == 0 and case["left"] >= 0:
                a = max(0, int(pos.min()) - case["left"])
            if case["op"] == "window" and case["right"] >= 0:
                e = min(n, max(case["sinks"], int(pos.max()) + case["right"] + 1))
            j = torch.arange(a, e, device="cuda")
            hide = None
            if case["op"] == "window":
                off = j[None, :] - pos[:, None]
                hide = torch.zeros_like(off, dtype=torch.bool)
                if case["left"] >= 0:
                    hide |= off < -case["left"]
                if case["right"] >= 0:
                    hide |= off > case["right"]
                hide &= j[None, :] >= case["sinks"]
            for h in range(Hq):
                z = torch.mm(s["q"][b, r0:r1, h].double(), keys[a:e, h // g].double().T) / math.sqrt(D)
                if hide is not None:
                    z = z.masked_fill(hide, -math.inf)
                out[b, r0:r1, h] = torch.mm(torch.softmax(z, 1).nan_to_num(0.0), values[a:e, h // g].double())
    return out
