"""Workloads of the operators around a GDN layer in a hybrid decoder: attention
of new tokens over a paged key-value cache, writing to that cache, evicting
from it, and the norms around a block.

``listed()`` names fixed cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` builds a case's inputs on the GPU, ``run`` makes one pass: in plain
torch operations where ``own`` is false, through this package's entry points
where it is true.  ``exact`` gives the results in 64 bits, ``work`` the bytes
and operations of a pass.
"""
import math

import torch

own = False

# Layers come as in the beam decode: heads of 64, 128 or 256, 256 beams that
# share a prompt of 1024 or 5120 tokens, up to 32 requests at a time.
_BEAM_STEPS = 7  # tokens each beam has of its own, the new one among them


def listed():
    return [
        # One short request, all in fp32: latency is all there is to it.
        dict(name="attn_one_short_f32", op="attention", R=1, W=1, H_q=4, H_kv=2, d=64, L=77, ragged=False,
             page=16, T=0, mass=False, dtype="f32"),
        # A batch of ordinary requests at very different lengths, one new token each.
        dict(name="attn_batch_ragged", op="attention", R=32, W=1, H_q=16, H_kv=4, d=128, L=5120, ragged=True,
             page=16, T=0, mass=False, dtype="bf16"),
        # Two long documents, with the attention weight of every token kept for eviction.
        dict(name="attn_long_mass", op="attention", R=2, W=1, H_q=32, H_kv=8, d=128, L=131000, ragged=False,
             page=64, T=0, mass=True, dtype="bf16"),
        # The wide beam decode: 256 beams on one 5120-token prompt.
        dict(name="attn_beams", op="attention", R=1, W=256, H_q=16, H_kv=4, d=128, L=5120, ragged=False,
             page=16, T=_BEAM_STEPS, mass=False, dtype="bf16"),
        # Several beam decodes at once on shorter prompts, large heads, with the weights.
        dict(name="attn_beams_batch_mass", op="attention", R=8, W=128, H_q=8, H_kv=2, d=256, L=1024, ragged=True,
             page=32, T=_BEAM_STEPS, mass=True, dtype="bf16"),
        # Each beam's new token, one per (request, beam).
        dict(name="write_beams", op="write", B=256, n=1, H_kv=4, d=128, start=6, page=1, dtype="bf16"),
        # A batch of prompts entering the cache.
        dict(name="write_prompts", op="write", B=8, n=5120, H_kv=8, d=128, start=0, page=16, dtype="bf16"),
        # A short cache halved.
        dict(name="evict_short", op="evict", R=1, H_kv=2, d=64, L=1000, keep=500, recent=64, page=16, dtype="f32"),
        # Long caches cut to an eighth.
        dict(name="evict_long", op="evict", R=8, H_kv=8, d=128, L=65500, keep=8192, recent=512, page=64,
             dtype="bf16"),
        # The gated per-head norm of one token's GDN output (fp32, as the decode step writes it).
        dict(name="norm_token_heads", op="norm", N=1, D=2048, group=128, y_dtype="f32", dtype="bf16", gate="silu",
             residual=False, scale=False, pre=False),
        # The beams of a decode step: post-norm, gate, residual scale and the next block's pre-norm.
        dict(name="norm_beams", op="norm", N=257, D=2048, group=2048, y_dtype="bf16", dtype="bf16", gate="sigmoid",
             residual=True, scale=True, pre=True),
        # Prompts of a batch through the same.
        dict(name="norm_prompts", op="norm", N=20480, D=4096, group=4096, y_dtype="bf16", dtype="bf16",
             gate="silu", residual=True, scale=True, pre=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "write", "evict", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 256, rng.randint(8, 256)])
    H_kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([1, 8, 16, 24, 32, 64])
    if op == "attention":
        G = rng.choice([1, 2, 3, 4, 8])
        if dtype == "bf16" and rng.random() < 0.5:  # beams on a shared prompt
            R, W, T = _log(rng, 1, 8), _log(rng, 2, 256), rng.randint(1, 12)
            L = _log(rng, 1, min(5120, max(1, 256 * 16 * 5120 * 128 // (R * W * G * H_kv * d))))
        else:
            R, W, T = _log(rng, 1, 32), 1, rng.choice([0, 0, 3])
            L = _log(rng, 1, 131000 * 2 * 8 * 128 // (R * H_kv * max(d, 128) * (2 if dtype == "f32" else 1)))
            L = min(L, 262000 // R)
        return dict(op=op, R=R, W=W, H_q=H_kv * G, H_kv=H_kv, d=d, L=L, ragged=rng.random() < 0.6, page=page, T=T,
                    mass=rng.random() < 0.4, dtype=dtype)
    if op == "write":
        B = _log(rng, 1, 256)
        n = _log(rng, 1, 40960 // (B * (2 if d > 128 else 1) * (2 if dtype == "f32" else 1)))
        return dict(op=op, B=B, n=n, H_kv=H_kv, d=d, start=rng.choice([0, rng.randint(0, 300)]), page=page, dtype=dtype)
    if op == "evict":
        R = _log(rng, 1, 8)
        L = _log(rng, 2, 65500 // ((2 if d > 128 else 1) * (2 if dtype == "f32" else 1)))
        keep = _log(rng, 1, max(1, min(L, 8192)))
        return dict(op=op, R=R, H_kv=H_kv, d=d, L=L, keep=keep, recent=rng.randint(0, keep), page=page, dtype=dtype)
    D, group = d * H_kv * 2, d
    if rng.random() < 0.5:
        D = _log(rng, 16, 8192)
        group = D
    residual = rng.random() < 0.7
    return dict(op=op, N=_log(rng, 1, min(20480, 20480 * 2048 // D)), D=D, group=group,
                y_dtype=rng.choice(["f32", "bf16"]), dtype=dtype, gate=rng.choice(["none", "sigmoid", "silu"]),
                residual=residual, scale=rng.random() < 0.5, pre=residual)


_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lengths(c):
    """Prompt lengths of the requests: all L, or spread up to it, the shortest L / R."""
    R, L = c["R"], c["L"]
    return [L * (r + 1) // R if c.get("ragged") else L for r in range(R)]


def _pool(gen, pages, H, page, d, dt):
    return torch.randn((pages, H, page, d), generator=gen, device="cuda", dtype=dt)


def _table(gen, rows, row_pages, pages):
    """Each row's pages, scattered over the pool; no page twice."""
    perm = torch.randperm(pages, generator=gen, device="cuda")[: rows * row_pages]
    return perm.to(torch.int32).reshape(rows, row_pages)


def prepare(case, seed):
    c, dt = case, _DT[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "attention":
        R, W, H, d, page, T = c["R"], c["W"], c["H_kv"], c["d"], c["page"], c["T"]
        row_pages = -(-c["L"] // page) + 1
        pages = R * row_pages + 3
        s["k"], s["v"] = _pool(gen, pages, H, page, d, dt), _pool(gen, pages, H, page, d, dt)
        s["table"] = _table(gen, R, row_pages, pages)
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        # Scores of standard deviation 2: a few tokens carry much of the weight.
        s["q"] = (2.0 * torch.randn((R, W, c["H_q"], d), generator=gen, device="cuda")).to(dt)
        s["scale"] = d ** -0.5
        if T:
            # Tokens of the beam tree, one page each, level by level; a beam's
            # table lists its ancestors by level and itself last.
            s["bk"], s["bv"] = _pool(gen, T * R * W, H, 1, d, dt), _pool(gen, T * R * W, H, 1, d, dt)
            parent = torch.randint(0, W, (T, R, W), generator=gen, device="cuda")
            first = (torch.arange(R, device="cuda") * W)[:, None]
            path = torch.arange(W, device="cuda").repeat(R, 1)
            at = []
            for level in reversed(range(T)):
                at.insert(0, level * R * W + first + path)
                path = torch.gather(parent[level], 1, path)
            s["btable"] = torch.stack(at, -1).to(torch.int32)
            s["blengths"] = torch.full((R, W), T, dtype=torch.int32, device="cuda")
        if c["mass"]:
            s["mass"] = torch.rand((R, H, row_pages * page), generator=gen, device="cuda")
            s["mass_out"] = torch.zeros_like(s["mass"])
    elif c["op"] == "write":
        B, n, H, d, page = c["B"], c["n"], c["H_kv"], c["d"], c["page"]
        row_pages = -(-(c["start"] + n) // page)
        pages = B * row_pages + 2
        s["k"] = torch.randn((B, n, H, d), generator=gen, device="cuda").to(dt)
        s["v"] = torch.randn((B, n, H, d), generator=gen, device="cuda").to(dt)
        s["k_pool"] = torch.zeros((pages, H, page, d), dtype=dt, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["table"] = _table(gen, B, row_pages, pages)
        s["start"] = torch.full((B,), c["start"], dtype=torch.int32, device="cuda")
    elif c["op"] == "evict":
        R, H, d, page, L, keep = c["R"], c["H_kv"], c["d"], c["page"], c["L"], c["keep"]
        row_pages, new_pages = -(-L // page), -(-keep // page)
        s["k"] = _pool(gen, R * row_pages, H, page, d, dt)
        s["v"] = _pool(gen, R * row_pages, H, page, d, dt)
        s["table"] = _table(gen, R, row_pages, R * row_pages)
        s["lengths"] = torch.full((R,), L, dtype=torch.int32, device="cuda")
        # Weights over several decades, and tokens that never drew any.
        m = torch.exp(2.5 * torch.randn((R, H, row_pages * page), generator=gen, device="cuda"))
        s["mass"] = torch.where(torch.rand(m.shape, generator=gen, device="cuda") < 0.1, torch.zeros_like(m), m)
        s["k2"] = torch.zeros((R * new_pages, H, page, d), dtype=dt, device="cuda")
        s["v2"] = torch.zeros_like(s["k2"])
        s["table2"] = _table(gen, R, new_pages, R * new_pages)
        s["mass2"] = torch.zeros((R, H, new_pages * page), device="cuda")
        s["lengths2"] = torch.zeros((R,), dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((R, H, keep), dtype=torch.int32, device="cuda")
    else:
        N, D = c["N"], c["D"]
        s["y"] = (0.3 * torch.randn((N, D), generator=gen, device="cuda")).to(_DT[c["y_dtype"]])
        s["w_post"] = 1.0 + 0.1 * torch.randn((c["group"],), generator=gen, device="cuda")
        if c["gate"] != "none":
            s["gate"] = torch.randn((N, D), generator=gen, device="cuda").to(dt)
        if c["residual"]:
            s["x"] = torch.randn((N, D), generator=gen, device="cuda").to(dt)
        if c["scale"]:
            s["scale"] = 0.2 * torch.randn((D,), generator=gen, device="cuda")
        if c["pre"]:
            s["w_pre"] = 1.0 + 0.1 * torch.randn((D,), generator=gen, device="cuda")
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    import linear_attention_beam_shared_b200 as L
    c = s["case"]
    if c["op"] == "attention":
        beam = (s["bk"], s["bv"], s["btable"], s["blengths"]) if c["T"] else None
        o = L.onela_paged_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], beam=beam, scale=s["scale"],
                                    mass=s.get("mass"), mass_out=s.get("mass_out"))
        return {"o": o, "mass": s["mass_out"]} if c["mass"] else {"o": o}
    if c["op"] == "write":
        L.onela_cache_write(s["k"], s["v"], s["k_pool"], s["v_pool"], s["table"], s["start"])
        return {"k": s["k_pool"], "v": s["v_pool"]}
    if c["op"] == "evict":
        L.onela_cache_evict(s["k"], s["v"], s["table"], s["lengths"], s["mass"], c["keep"], c["recent"], s["k2"],
                            s["v2"], s["table2"], s["lengths2"], s["mass2"], kept=s["kept"])
        return {"k": s["k2"], "v": s["v2"], "mass": s["mass2"], "lengths": s["lengths2"], "kept": s["kept"]}
    x_out, n_out = L.onela_block_norm(
        s["y"], x=s.get("x"), gate=s.get("gate"), gate_act=c["gate"], w_post=s["w_post"], scale=s.get("scale"),
        alpha=0.5, w_pre=s.get("w_pre"), eps=1e-6, dtype=c["dtype"])
    return {"x": x_out, "n": n_out} if c["pre"] else {"x": x_out}


# ---------------------------------------------------------------- plain forms

def _rows(pool, table):
    """[pages][H][page][d] through a table [R][P] to fp32 [R][H][P page][d]."""
    t = pool[table.long()].float()
    return t.transpose(1, 2).reshape(t.shape[0], t.shape[2], -1, t.shape[-1])


def _attention(s):
    c = s["case"]
    R, W, H, d = c["R"], c["W"], c["H_kv"], c["d"]
    G = c["H_q"] // H
    k, v = _rows(s["k"], s["table"]), _rows(s["v"], s["table"])
    q = s["q"].float().reshape(R, W, H, G, d).permute(0, 2, 1, 3, 4)      # [R][H][W][G][d]
    n = k.shape[2]
    live = torch.arange(n, device="cuda")[None] < s["lengths"][:, None]
    v = torch.where(live[:, None, :, None], v, torch.zeros((), device="cuda"))
    sc = (q.reshape(R, H, W * G, d) @ k.transpose(2, 3)) * s["scale"]
    sc = sc.masked_fill(~live[:, None, None, :], -math.inf).reshape(R, H, W, G, n)
    if c["T"]:
        bk = s["bk"][s["btable"].long()].float()[:, :, :, :, 0].permute(0, 3, 1, 2, 4)   # [R][H][W][T][d]
        bv = s["bv"][s["btable"].long()].float()[:, :, :, :, 0].permute(0, 3, 1, 2, 4)
        bs = (q @ bk.transpose(3, 4)) * s["scale"]
        bl = torch.arange(c["T"], device="cuda")[None, None] < s["blengths"][:, :, None]
        sc = torch.cat([sc, bs.masked_fill(~bl[:, None, :, None, :], -math.inf)], -1)
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    p = e / e.sum(-1, keepdim=True).clamp_min(1e-38)
    o = (p[..., :n].reshape(R, H, W * G, n) @ v).reshape(R, H, W, G, d)
    if c["T"]:
        o = o + p[..., n:] @ bv
    out = {"o": o.permute(0, 2, 1, 3, 4).reshape(R, W, c["H_q"], d).to(s["q"].dtype)}
    if c["mass"]:
        drawn = s["mass"] + p[..., :n].sum((2, 3))
        s["mass_out"].copy_(torch.where(live[:, None], drawn, s["mass_out"]))
        out["mass"] = s["mass_out"]
    return out


def _write(s):
    c = s["case"]
    pos = s["start"].long()[:, None] + torch.arange(c["n"], device="cuda")
    page = torch.gather(s["table"].long(), 1, pos // c["page"])
    s["k_pool"][page, :, pos % c["page"]] = s["k"]
    s["v_pool"][page, :, pos % c["page"]] = s["v"]
    return {"k": s["k_pool"], "v": s["v_pool"]}


def _evict(s):
    c = s["case"]
    R, H, L, page = c["R"], c["H_kv"], c["L"], c["page"]
    n = min(L, c["keep"])
    m = s["mass"][:, :, :L]
    recent = torch.arange(L, device="cuda") >= L - c["recent"]
    order = torch.argsort(torch.where(recent, math.inf, m), dim=-1, descending=True, stable=True)
    kept = torch.sort(order[..., :n], dim=-1).values                                    # [R][H][n]
    head = torch.arange(H, device="cuda")[None, :, None]
    src = torch.gather(s["table"].long()[:, None].expand(R, H, -1), 2, kept // page)
    to = torch.arange(n, device="cuda")
    dst = s["table2"].long()[:, None, to // page].expand(R, H, n)
    s["k2"][dst, head, to % page] = s["k"][src, head, kept % page]
    s["v2"][dst, head, to % page] = s["v"][src, head, kept % page]
    s["mass2"][:, :, :n] = torch.gather(m, 2, kept)
    s["lengths2"].copy_(s["lengths"].clamp_max(c["keep"]))
    s["kept"][:, :, :n] = kept.to(torch.int32)
    return {"k": s["k2"], "v": s["v2"], "mass": s["mass2"], "lengths": s["lengths2"], "kept": s["kept"]}


def _norm(s):
    c = s["case"]
    N, D, dt = c["N"], c["D"], _DT[c["dtype"]]
    y = s["y"].float().reshape(N, D // c["group"], c["group"])
    u = (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s["w_post"]).reshape(N, D)
    if c["gate"] != "none":
        z = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        u = u * (z * sig if c["gate"] == "silu" else sig)
    u = 0.5 * u
    if c["scale"]:
        u = u * s["scale"]
    x = u + s["x"].float() if c["residual"] else u
    out = {"x": x.to(dt)}
    if c["pre"]:
        out["n"] = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["w_pre"]).to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"attention": _attention, "write": _write, "evict": _evict, "norm": _norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------- bytes, operations, exact results

def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "attention":
        rows, n = c["W"] * c["H_q"], sum(_lengths(c))
        own_tokens = c["R"] * c["W"] if c["T"] else 0  # of the beam tree at least every beam's new token
        b = (n + own_tokens) * c["H_kv"] * c["d"] * 2 * es + 2 * c["R"] * rows * c["d"] * es
        b += 4 * (n // c["page"] + c["R"] * (1 + c["W"] * c["T"]))
        if c["mass"]:
            b += 8 * c["H_kv"] * n
        return {"bytes": b, "flops": 4 * c["d"] * rows * (n + c["R"] * c["T"])}
    if c["op"] == "write":
        return {"bytes": 4 * c["B"] * c["n"] * c["H_kv"] * c["d"] * es + 4 * c["B"] * (1 + c["n"] // c["page"]),
                "flops": 0}
    if c["op"] == "evict":
        n = min(c["L"], c["keep"])
        per_head = 4 * c["L"] + n * (4 * c["d"] * es + 4 + 4)
        return {"bytes": c["R"] * (c["H_kv"] * per_head + 8 + 4 * (c["L"] + n) // c["page"]), "flops": 0}
    parts = (4 if c["y_dtype"] == "f32" else 2) + es * (
        (c["gate"] != "none") + c["residual"] + 1 + c["pre"])
    return {"bytes": c["N"] * c["D"] * parts + 4 * (c["group"] + c["D"] * (c["scale"] + c["pre"])),
            "flops": 12 * c["N"] * c["D"]}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "write":
        return _exact_write(c, s)
    if c["op"] == "evict":
        return _exact_evict(c, s)
    return _exact_norm(c, s)


def _tokens(pool, row, n, page):
    """The n tokens of one table row in 64 bits, [H][n][d]."""
    j = torch.arange(n, device="cuda")
    return pool[row.long()[j // page], :, j % page].double().transpose(0, 1)


def _exact_attention(c, s):
    R, W, H, d, page, T = c["R"], c["W"], c["H_kv"], c["d"], c["page"], c["T"]
    G = c["H_q"] // H
    o = torch.zeros((R, W, H, G, d), dtype=torch.float64, device="cuda")
    mass = s["mass_out"].double() if c["mass"] else None
    for r, n in enumerate(_lengths(c)):
        k, v = _tokens(s["k"], s["table"][r], n, page), _tokens(s["v"], s["table"][r], n, page)
        for h in range(H):
            q = s["q"][r].double().reshape(W, H, G, d)[:, h]                     # [W][G][d]
            logit = torch.einsum("wgd,nd->wgn", q, k[h]) * s["scale"]
            if T:
                at = s["btable"][r].long()                                       # [W][T]
                bk, bv = s["bk"][at, h, 0].double(), s["bv"][at, h, 0].double()  # [W][T][d]
                logit = torch.cat([logit, torch.einsum("wgd,wtd->wgt", q, bk) * s["scale"]], -1)
            if not logit.shape[-1]:
                continue
            w = torch.exp(logit - torch.logsumexp(logit, -1, keepdim=True))
            o[r, :, h] = torch.einsum("wgn,nd->wgd", w[..., :n], v[h])
            if T:
                o[r, :, h] += torch.einsum("wgt,wtd->wgd", w[..., n:], bv)
            if mass is not None:
                mass[r, h, :n] = s["mass"][r, h, :n].double() + w[..., :n].sum((0, 1))
    out = {"o": o.reshape(R, W, c["H_q"], d)}
    return {**out, "mass": mass} if c["mass"] else out


def _exact_write(c, s):
    out = {"k": s["k_pool"].double(), "v": s["v_pool"].double()}
    n, page = c["n"], c["page"]
    j = c["start"] + torch.arange(n, device="cuda")
    for b in range(c["B"]):
        at = s["table"][b].long()[j // page]
        out["k"][at, :, j % page] = s["k"][b].double()
        out["v"][at, :, j % page] = s["v"][b].double()
    return out


def _exact_evict(c, s):
    L, page = c["L"], c["page"]
    n, free = min(L, c["keep"]), max(L - c["recent"], 0)
    k2, v2, mass2 = s["k2"].double(), s["v2"].double(), s["mass2"].double()
    kept_all = s["kept"].clone()
    to = torch.arange(n, device="cuda")
    for r in range(c["R"]):
        dst = s["table2"][r].long()[to // page]
        for h in range(c["H_kv"]):
            m = s["mass"][r, h, :L].double()
            last = torch.arange(free, L, device="cuda")
            best = torch.sort(m[:free], descending=True, stable=True).indices[: n - min(n, len(last))]
            kept = torch.cat([best, last[len(last) - min(n, len(last)):]]).sort().values
            src = s["table"][r].long()[kept // page]
            k2[dst, h, to % page] = s["k"][src, h, kept % page].double()
            v2[dst, h, to % page] = s["v"][src, h, kept % page].double()
            mass2[r, h, :n] = m[kept]
            kept_all[r, h, :n] = kept.to(torch.int32)
    return {"k": k2, "v": v2, "mass": mass2, "lengths": torch.full_like(s["lengths"], n), "kept": kept_all}


def _exact_norm(c, s):
    N, D, g = c["N"], c["D"], c["group"]
    u = s["y"].double()
    power = u.square().reshape(N, D // g, g).sum(-1) / g
    u = u / torch.sqrt(power + 1e-6).repeat_interleave(g, 1) * s["w_post"].double().repeat(D // g)
    if c["gate"] != "none":
        z = s["gate"].double()
        u = u * torch.sigmoid(z) * (z if c["gate"] == "silu" else 1.0)
    x = 0.5 * u * (s["scale"].double() if c["scale"] else 1.0)
    if c["residual"]:
        x = x + s["x"].double()
    out = {"x": x}
    if c["pre"]:
        out["n"] = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6) * s["w_pre"].double()
    return out
