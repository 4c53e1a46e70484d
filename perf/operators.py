"""Cases of the paged serving operators: norms of queries and keys with the position
rotation, append to a paged key-value cache, decode over the pages, and decode over the
pages that a cheap score selects.  Each has its plain form (elementary torch operations),
its inputs and its definition in 64 bits.

Cache layout: keys [page][kv head][d/16][slot][16] (rotated, interleaved pairs, 8-pair
chunks), values [page][kv head][slot][d], bounds [page][kv head][2][d] (elementwise
minimum and maximum of the page's keys).
"""
import math
import random

import torch

own = False

THETA = 1e7


def _case(name, op, **kw):
    """A case with every field present (the unused ones at neutral values)."""
    c = dict(name=name, op=op, batch=1, tokens=1, max_len=0, ragged=False, heads=28, kv_heads=4, d=128, page=64,
             theta=THETA, alpha=1.0, dtype="bf16", norm=True, axes=1, rotate_half=True, n_select=0)
    c.update(kw)
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # the queries and keys of one 8192-token prompt, normed and rotated ahead of the prefill
        _case("norm_rope_8k", "norm_rope", tokens=8192),
        # a small full-precision model over image patches: three position axes, odd token count
        _case("norm_rope_axes_fp32", "norm_rope", tokens=1111, heads=4, kv_heads=4, d=64, theta=1e4, dtype="fp32",
              axes=3, rotate_half=False),
        # one user, one new token: the call's latency
        _case("append_step_1", "append", batch=1, max_len=700, page=16),
        # a full serving batch, one new token each
        _case("append_step_256", "append", batch=256, max_len=1024, ragged=True),
        # ragged prompts behind cached prefixes, image positions, large pages
        _case("append_prompts_32k", "append", batch=5, tokens=32768, max_len=3000, ragged=True, page=128, axes=3),
        # one short sequence of a small model: latency
        _case("decode_short", "decode", batch=1, max_len=777, heads=4, kv_heads=4, d=64, page=16, theta=1e4),
        # one user at 131072 tokens
        _case("decode_128k", "decode", batch=1, max_len=131072),
        # a ragged serving batch (one row is padding), small pages
        _case("decode_batch_64", "decode", batch=64, max_len=8192, ragged=True, page=16),
        # four caches of 1048576 tokens, large pages
        _case("decode_4x1m", "decode", batch=4, max_len=1 << 20, page=128),
        # one user at 1048576 tokens who attends to 64 pages of 64
        _case("select_1m", "select", batch=1, max_len=1 << 20, n_select=64),
        # a ragged batch without windows
        _case("select_batch_32", "select", batch=32, max_len=32768, ragged=True, page=32, alpha=0.0, n_select=48),
        # short caches of a small model: latency
        _case("select_short", "select", batch=8, max_len=4000, heads=14, kv_heads=2, d=64, page=16, n_select=20,
              ragged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "append", "decode", "decode", "select", "select"])
    kvh = rng.choice([1, 2, 3, 4, 8])
    c = dict(heads=kvh * rng.randint(1, 8), kv_heads=kvh, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             theta=rng.choice([1e4, 5e5, 1e7]), alpha=rng.choice([0.0, 0.5, 1.0, 1.0]),
             rotate_half=rng.random() < 0.6, norm=rng.random() < 0.8, axes=rng.choice([1, 1, 2, 3]),
             ragged=rng.random() < 0.7)
    if op == "norm_rope":
        c.update(tokens=_log_int(rng, 1, 20000), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    elif op == "append":
        c["batch"] = _log_int(rng, 1, 300)
        c["max_len"] = _log_int(rng, 1, 2000)
        c["tokens"] = 1 if rng.random() < 0.5 else _log_int(rng, c["batch"] + 1, 20000)
    else:
        c["batch"] = _log_int(rng, 1, 200)
        c["max_len"] = _log_int(rng, 1, max(2, min(1 << 20, (1 << 21) // (c["batch"] * kvh))))
        if op == "select":
            c["n_select"] = _log_int(rng, 2, 96)
    return _case(None, op, **c)


# ------------------------------------------------------------------ sizes of a case

def _lengths(c):
    """Cached tokens of each sequence (they belong to the case, not to the seed)."""
    r = random.Random("%d %d %d" % (c["batch"], c["max_len"], c["page"]))
    if not c["ragged"]:
        return [c["max_len"]] * c["batch"]
    n = [r.randint(1, c["max_len"]) for _ in range(c["batch"])]
    n[0] = c["max_len"]
    if c["batch"] >= 4:
        n[c["batch"] // 2] = 0  # a padding row of the batch, or a sequence without a cache
    return n


def _new_tokens(c):
    """New tokens of each sequence of an append."""
    if c["tokens"] <= 1:
        return [1] * c["batch"]
    r = random.Random("%d %d" % (c["batch"], c["tokens"]))
    cut = sorted(r.randint(0, c["tokens"]) for _ in range(c["batch"] - 1))
    return [b - a for a, b in zip([0] + cut, cut + [c["tokens"]])]


def _windows(c):
    """Largest distance at which each pair still counts."""
    lam = [2 * math.pi * c["theta"] ** (2.0 * i / c["d"]) for i in range(c["d"] // 2)]
    return [min(2 ** 31 - 1, math.ceil(c["alpha"] * x)) if c["alpha"] else 2 ** 31 - 1 for x in lam]


def _axis_of_pair(c):
    """Position axis of each pair: contiguous sections, the first the smallest."""
    n, a = c["d"] // 2, c["axes"]
    return [0] * n if a == 1 else [0] * (n // 4) + [1 + (j * (a - 1)) // (n - n // 4) for j in range(n - n // 4)]


def work(case):
    c = case
    H, Hkv, d = c["heads"], c["kv_heads"], c["d"]
    if c["op"] == "norm_rope":
        rows, esz = c["tokens"] * (H + Hkv), 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * rows * d * esz + c["tokens"] * 8 * c["axes"], "flops": 8 * rows * d}
    if c["op"] == "append":
        new, old = _new_tokens(c), _lengths(c)
        T = sum(new)
        pages = sum((s + n - 1) // c["page"] - s // c["page"] + 1 for s, n in zip(old, new) if n)
        part = sum(1 for s, n in zip(old, new) if n and s % c["page"])
        return {"bytes": 2 * T * (H + 2 * Hkv) * d * 2 + T * 8 * (c["axes"] if c["axes"] > 1 else 0)
                + (pages + part) * Hkv * 4 * d, "flops": 8 * T * (H + Hkv) * d}
    lens, W, ps = _lengths(c), _windows(c), c["page"]
    active = sum(min(n, w + 1) for n in lens for w in W)  # (key, pair) within the windows
    keys = sum(lens)
    io = 4 * len(lens) * H * d + sum(4 * -(-n // ps) for n in lens)
    if c["op"] == "decode":
        return {"bytes": active * Hkv * 4 + keys * Hkv * d * 2 + io, "flops": 4 * active * H + 2 * keys * H * d}
    pages = [-(-n // ps) for n in lens]
    kept = sum(min(n, c["n_select"] * ps) for n in lens)
    share = active / max(1, keys * d // 2)
    return {"bytes": sum(pages) * Hkv * 4 * d + kept * Hkv * d * 2 * (1 + share) + io + 4 * len(lens) * Hkv * c["n_select"],
            "flops": 3 * sum(pages) * H * d + kept * H * d * 2 * (1 + share)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    c = case
    H, Hkv, d, ps, B = c["heads"], c["kv_heads"], c["d"], c["page"], c["batch"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    s = dict(case=c, windows=torch.tensor(_windows(c), device="cuda"), axis=_axis_of_pair(c),
             axis_index=torch.tensor(_axis_of_pair(c), device="cuda"),
             omega=torch.tensor([c["theta"] ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda"))
    if c["op"] in ("norm_rope", "append"):
        new = _new_tokens(c) if c["op"] == "append" else [c["tokens"]]
        T = sum(new)
        # one row per token of the fused projection: queries, keys, values
        qkv = normal(T, (H + 2 * Hkv) * d, dtype=dt)
        s["q"] = qkv[:, :H * d].view(T, H, d)
        s["k"] = qkv[:, H * d:(H + Hkv) * d].view(T, Hkv, d)
        s["v"] = qkv[:, (H + Hkv) * d:].view(T, Hkv, d)
        s["q_weight"] = (1 + normal(d, dtype=torch.float32, std=0.1)).to(dt) if c["norm"] else None
        s["k_weight"] = (1 + normal(d, dtype=torch.float32, std=0.1)).to(dt) if c["norm"] else None
        s["eps"] = 1e-6
        s["q_out"] = torch.empty((T, H, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((T, Hkv, d), dtype=dt, device="cuda")
        first = _lengths(c) if c["op"] == "append" else [0]
        n, off = torch.tensor(new, device="cuda"), torch.tensor(first, device="cuda")
        cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
        s["seq"] = torch.repeat_interleave(torch.arange(len(new), device="cuda"), n)
        t = torch.arange(T, device="cuda") - cu[s["seq"]]
        s["slot"] = off[s["seq"]] + t
        s["pos"] = None if c["op"] == "append" and c["axes"] == 1 else s["slot"][None].contiguous()
        if c["axes"] > 1:  # image patches: time, then the row and column of a 36-wide picture
            more = [s["slot"] // 1296, s["slot"] % 1296 // 36, s["slot"] % 36]
            s["pos"] = torch.stack([x + off[s["seq"]] for x in more[3 - c["axes"]:]]).contiguous()
        s["start"] = off.to(torch.int32)
        s["cu"] = None if c["tokens"] <= 1 else cu.to(torch.int32)
        after = [a + b for a, b in zip(first, new)]
    else:
        after = _lengths(c)
        s["q"] = normal(B, H, d, std=2.0)
        s["out"] = torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((B, H), dtype=torch.float32, device="cuda")
        s["kv_len"] = torch.tensor(after, dtype=torch.int32, device="cuda")
    if c["op"] == "norm_rope":
        return s
    # a pool of pages and each sequence's pages in it, in no order
    counts = [-(-n // ps) for n in after]
    total, most = sum(counts), max(1, max(counts))
    pool = total + 3
    order = torch.randperm(pool, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(most, device="cuda")[None] < torch.tensor(counts, device="cuda")[:, None]] = order
    s["page_table"] = table
    s["k_pages"] = normal(pool, Hkv, d // 16, ps, 16)
    s["v_pages"] = normal(pool, Hkv, ps, d)
    if c["op"] == "select":  # keys of a page lie together, as keys of neighbouring tokens do
        s["k_pages"] += normal(pool, Hkv, d // 16, 1, 16)
        s["selected"] = torch.empty((B, Hkv, c["n_select"]), dtype=torch.int32, device="cuda")
    if c["op"] in ("append", "select"):
        s["bounds"] = torch.stack([s["k_pages"].amin(3).view(pool, Hkv, d), s["k_pages"].amax(3).view(pool, Hkv, d)], 2)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from rope_frequency_sparse_b200 import atf

    c = s["case"]
    pairing = atf.ATF_PAIRS_ROTATE_HALF if c["rotate_half"] else atf.ATF_PAIRS_INTERLEAVED
    alpha = c["alpha"] or math.inf
    if c["op"] == "norm_rope":
        q, k = atf.qk_norm_rope(s["q"], s["k"], c["theta"], s["pos"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                eps=s["eps"], pair_axis=s["axis"], pairing=pairing, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    if c["op"] == "append":
        q = atf.paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["start"], c["theta"],
                             cu=s["cu"], pos=s["pos"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                             pair_axis=s["axis"], pairing=pairing, bounds=s["bounds"], q_out=s["q_out"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "bounds": s["bounds"]}
    if "workspace" not in s:  # a serving loop keeps its scratch
        need = atf.atf_paged_decode_workspace_bytes(c["batch"], c["heads"], c["kv_heads"], c["d"])
        if c["op"] == "select":
            need = max(need, atf.atf_page_select_workspace_bytes(c["batch"], c["kv_heads"], s["page_table"].shape[1]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if c["op"] == "decode":
        out = atf.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], c["theta"], alpha,
                               lse=s["lse"], out=s["out"], workspace=s["workspace"])
        return {"out": out, "lse": s["lse"]}
    sel = atf.page_select(s["q"], s["bounds"], s["page_table"], s["kv_len"], c["page"], c["n_select"], c["theta"], alpha,
                          n_first=1, n_last=1, selected=s["selected"], workspace=s["workspace"])
    out = atf.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], c["theta"], alpha,
                           selected=sel, out=s["out"], workspace=s["workspace"])
    return {"selected": sel, "out": out}


def _norm_rope(s, x, weight):
    """Each head normed, then each pair turned by its axis' position; pairs written interleaved."""
    c = s["case"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    pos = s["pos"] if s["pos"] is not None else s["slot"][None]
    ang = pos[s["axis_index"]].double().T * s["omega"]  # angles of far positions need 64 bits
    cs, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = y.chunk(2, -1) if c["rotate_half"] else (y[..., 0::2], y[..., 1::2])
    return torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2).to(x.dtype)


def _attend(s, logical):
    """Softmax attention over the given pages [batch][kv head][n] (-1: none), and its log of sums."""
    c, ps = s["case"], s["case"]["page"]
    B, H, d = s["q"].shape
    Hkv = c["kv_heads"]
    rows = torch.arange(B, device="cuda")[:, None, None]
    page = s["page_table"][rows, logical.clamp(min=0)].clamp(min=0).long()
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    key = logical[..., None] * ps + torch.arange(ps, device="cuda")
    last = s["kv_len"].long()[:, None, None, None] - 1
    live = ((key <= last) & (logical >= 0)[..., None]).flatten(2)  # [B][Hkv][n * ps]
    K = s["k_pages"][page, head].permute(0, 1, 2, 4, 3, 5).float().reshape(B, Hkv, -1, d // 2, 2)
    K = K * ((last - key).flatten(2)[..., None] <= s["windows"])[..., None]  # pairs beyond their window
    V = s["v_pages"][page, head].float().reshape(B, Hkv, -1, d)
    K = K.flatten(3).masked_fill(~live[..., None], 0.0)
    V = V.masked_fill(~live[..., None], 0.0)
    x = s["q"].float().view(B, Hkv, H // Hkv, d) @ K.transpose(2, 3) / math.sqrt(d)
    x = x.masked_fill(~live[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    out = p @ V / total.clamp(min=1e-30)
    return out.reshape(B, H, d).to(s["q"].dtype), (total.log() + top).masked_fill(total == 0, -math.inf).reshape(B, H)


def _select(s):
    """The pages with the highest bound on a logit; 64-bit sums, since neighbours in rank are close."""
    c, ps = s["case"], s["case"]["page"]
    B, H, d = s["q"].shape
    P, Hkv, n = s["page_table"].shape[1], c["kv_heads"], c["n_select"]
    b = s["bounds"][s["page_table"].clamp(min=0).long()].double()  # [B][P][Hkv][2][d]
    q = s["q"].double().view(B, 1, Hkv, H // Hkv, d)
    term = torch.maximum(q * b[:, :, :, None, 0], q * b[:, :, :, None, 1])
    index, length = torch.arange(P, device="cuda"), s["kv_len"].long()[:, None]
    pages = (length + ps - 1) // ps
    nearest = length - 1 - torch.minimum(index * ps + ps - 1, length - 1)  # [B][P]
    on = nearest[..., None] <= s["windows"]
    score = (term.view(B, P, Hkv, H // Hkv, d // 2, 2).sum(-1) * on[:, :, None, None]).sum(-1).amax(-1).transpose(1, 2)
    forced = (index < 1) | (index >= pages - 1)
    score = score.masked_fill(forced[:, None], math.inf).masked_fill((index >= pages)[:, None], -math.inf)
    kept = score.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    kept = kept.masked_fill(kept >= pages[..., None], P).sort(-1).values
    kept = torch.nn.functional.pad(kept, (0, n - kept.shape[-1]), value=P)
    return kept.masked_fill(kept == P, -1)


def _run_plain(s):
    c, ps = s["case"], s["case"]["page"]
    if c["op"] == "norm_rope":
        return {"q": _norm_rope(s, s["q"], s["q_weight"]), "k": _norm_rope(s, s["k"], s["k_weight"])}
    if c["op"] == "append":
        k, v = _norm_rope(s, s["k"], s["k_weight"]), s["v"]
        page, at = s["page_table"][s["seq"], s["slot"] // ps].long(), s["slot"] % ps
        T, Hkv, d = k.shape
        s["k_pages"][page, :, :, at] = k.view(T, Hkv, d // 16, 16)
        s["v_pages"][page, :, at] = v
        # a page that held no keys before starts its bounds anew
        index = page[:, None, None].expand(T, Hkv, d)
        fresh = page[at == 0]
        low, high = s["bounds"][:, :, 0].float(), s["bounds"][:, :, 1].float()
        low[fresh], high[fresh] = math.inf, -math.inf
        low.scatter_reduce_(0, index, k.float(), "amin")
        high.scatter_reduce_(0, index, k.float(), "amax")
        s["bounds"][:, :, 0], s["bounds"][:, :, 1] = low, high
        return {"q": _norm_rope(s, s["q"], s["q_weight"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"],
                "bounds": s["bounds"]}
    if c["op"] == "decode":
        every = torch.arange(s["page_table"].shape[1], device="cuda").expand(c["batch"], c["kv_heads"], -1)
        out, lse = _attend(s, every)
        return {"out": out, "lse": lse}
    sel = _select(s)
    return {"selected": sel.to(torch.int32), "out": _attend(s, sel)[0]}


# ------------------------------------------------------------------ the definition in 64 bits

def _turned(x, weight, eps, angle, rotate_half):
    """x [T][H][d] as complex pairs, scaled and turned by exp(i angle) [T][d/2]."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt()
    half = x.shape[-1] // 2
    z = torch.complex(x[..., :half], x[..., half:]) if rotate_half else torch.view_as_complex(
        x.reshape(*x.shape[:-1], half, 2).contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.view_as_real(z).reshape(x.shape)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    ps, d, Hkv = c["page"], c["d"], c["kv_heads"]
    G = c["heads"] // Hkv
    if c["op"] in ("norm_rope", "append"):
        pos = s["pos"] if s["pos"] is not None else s["slot"][None]
        angle = torch.stack([pos[a].double() * c["theta"] ** (-2.0 * i / d) for i, a in enumerate(s["axis"])], 1)
        q, k = (_turned(s[n], s[n + "_weight"], s["eps"], angle, c["rotate_half"]) for n in "qk")
        if c["op"] == "norm_rope":
            return {"q": q, "k": k}
        kp, vp, bd = s["k_pages"].double(), s["v_pages"].double(), s["bounds"].double()
        slots, row = s["slot"].tolist(), 0
        for b, n in enumerate(_new_tokens(c)):
            t = row
            while t < row + n:  # the new tokens that fall into one page
                m = min(row + n - t, ps - slots[t] % ps)
                page, at = int(s["page_table"][b, slots[t] // ps]), slots[t] % ps
                kp[page, :, :, at:at + m] = k[t:t + m].reshape(m, Hkv, d // 16, 16).permute(1, 2, 0, 3)
                vp[page, :, at:at + m] = s["v"][t:t + m].double().transpose(0, 1)
                lo, hi = k[t:t + m].amin(0), k[t:t + m].amax(0)
                bd[page, :, 0] = torch.minimum(bd[page, :, 0], lo) if at else lo
                bd[page, :, 1] = torch.maximum(bd[page, :, 1], hi) if at else hi
                t += m
            row += n
        return {"q": q, "k_pages": kp, "v_pages": vp, "bounds": bd}
    lens = s["kv_len"].tolist()
    window = torch.tensor(_windows(c), device="cuda").repeat_interleave(2)
    out = torch.zeros(c["batch"], c["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    chosen = torch.full((c["batch"], Hkv, c["n_select"]), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        P = -(-n // ps)
        if not n:
            continue
        pages = s["page_table"][b, :P].long()
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            keep = torch.arange(P, device="cuda")
            if c["op"] == "select":
                lo, hi = s["bounds"][pages, h].double().unbind(1)
                near = (n - ps * (keep + 1)).clamp(min=0)  # distance of the page's last key
                on = (near[:, None] <= window).double()
                best = (q.clamp(min=0) @ (hi * on).T + q.clamp(max=0) @ (lo * on).T).amax(0)
                best[0] = best[-1] = math.inf
                order = sorted(range(P), key=lambda i, v=best.tolist(): (-v[i], i))[:c["n_select"]]
                keep = torch.tensor(sorted(order), device="cuda")
                chosen[b, h, :len(order)] = keep.to(torch.int32)
            key = (keep[:, None] * ps + torch.arange(ps, device="cuda")).flatten()
            key = key[key < n]
            page, at = pages[key // ps], key % ps
            K = s["k_pages"][page, h, :, at].double().flatten(1) * ((n - 1 - key)[:, None] <= window)
            x = q @ K.T * d ** -0.5
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ s["v_pages"][page, h, at].double()
    return {"out": out, "lse": lse} if c["op"] == "decode" else {"selected": chosen, "out": out}
