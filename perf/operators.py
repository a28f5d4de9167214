"""The operators around the Gated DeltaNet step of a hybrid layer, as cases to measure: the norms before and after a
block with its gate and residual scale, rotary positions, the page tables of a serving step, and the block attention of
the softmax layers over a paged cache whose requests share a prefix.

Each case is one call (or a forward with its reverse mode) as a user's program makes it.  `run` computes the plain
form of the operators with elementary torch operations in fp32, or, where `own` is set, calls the library.
"""
import math

import torch

own = False

# gate activations, as the library numbers them
LINEAR, SILU, SIGMOID = 0, 1, 2


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the serving step of 256 requests x 4 tokens: the GDN output's norm per head with its SiLU gate
        {"name": "gated_norm_step", "op": "gated_norm", "train": False, "T": 1024, "H": 16, "d": 128, "io": "bf16",
         "gate": True, "act": SILU},
        # the training step of 4 x 8192 tokens, forward and reverse mode, the gate a slice of a fused projection
        {"name": "gated_norm_train", "op": "gated_norm", "train": True, "T": 32768, "H": 16, "d": 128, "io": "bf16",
         "gate": True, "act": SILU},
        # an fp32 run with an odd head count and a head width that is no power of two
        {"name": "gated_norm_fp32_odd", "op": "gated_norm", "train": True, "T": 1531, "H": 5, "d": 72, "io": "f32",
         "gate": True, "act": SIGMOID},
        # one token of one request: only latency counts
        {"name": "residual_norm_token", "op": "residual_norm", "train": False, "T": 1, "C": 2048, "io": "bf16",
         "res": "bf16", "gate": False, "post": False, "scale": False, "act": LINEAR},
        # the training step: post-norm, gate, channel scale, fp32 residual stream, forward and reverse mode
        {"name": "residual_norm_train", "op": "residual_norm", "train": True, "T": 32768, "C": 2048, "io": "bf16",
         "res": "f32", "gate": True, "post": True, "scale": True, "act": SIGMOID},
        # packed training rows of the softmax layers, a quarter of each head rotated, q and k slices of one projection
        {"name": "rotary_train", "op": "rotary", "train": True, "T": 32768, "Hq": 16, "Hk": 4, "d": 128, "rot": 32,
         "inter": False, "far": 8192, "factor": 1.0, "io": "bf16"},
        # the serving step: 256 requests x 4 tokens far into a scaled context, keys and values into the cache
        {"name": "rotary_cache_step", "op": "rotary", "train": False, "T": 1024, "Hq": 16, "Hk": 4, "d": 128, "rot": 128,
         "inter": True, "far": 1000000, "factor": 8.0, "io": "bf16", "page": 64},
        # the tables of the same serving step: 256 requests, 4 new tokens each
        {"name": "step_tables_block", "op": "step_tables", "R": 256, "held": 1024, "new": 4, "ragged": False, "page": 64},
        # the tables of a prefill: 700 prompts of 0 to 2047 tokens
        {"name": "step_tables_prefill", "op": "step_tables", "R": 700, "held": 0, "new": 2047, "ragged": True, "page": 16},
        # one request, one token, a long cache of its own and no shared prefix
        {"name": "attention_token_long", "op": "attention", "R": 1, "B": 1, "Hk": 4, "G": 4, "d": 128, "prefix": 0,
         "own": 16384, "page": 64, "causal": False},
        # 256 requests x 4 tokens over a shared prefix of 8192 tokens and up to 1024 tokens each of their own
        {"name": "attention_shared_prefix", "op": "attention", "R": 256, "B": 4, "Hk": 4, "G": 4, "d": 128, "prefix": 8192,
         "own": 1024, "page": 64, "causal": False},
        # a draft of 7 tokens verified causally: 37 requests, odd prefix, small pages, wide heads
        {"name": "attention_verify_odd", "op": "attention", "R": 37, "B": 7, "Hk": 2, "G": 8, "d": 256, "prefix": 2500,
         "own": 777, "page": 16, "causal": True},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_norm", "residual_norm", "rotary", "step_tables", "attention"])
    io = rng.choice(["bf16", "bf16", "f32"])
    act = rng.choice([LINEAR, SILU, SIGMOID])
    if op == "gated_norm":
        H, d = rng.randint(1, 32), rng.choice([16, 64, 72, 128, 192, 256, rng.randint(1, 300)])
        T = _log(rng, 1, min(32768, (1 << 25) // (H * d)))
        return {"op": op, "train": rng.random() < 0.5, "T": T, "H": H, "d": d, "io": io, "gate": rng.random() < 0.8,
                "act": act}
    if op == "residual_norm":
        C = rng.choice([16 * rng.randint(1, 512), _log(rng, 1, 8192)])
        T = _log(rng, 1, min(32768, (1 << 25) // C))
        return {"op": op, "train": rng.random() < 0.5, "T": T, "C": C, "io": io,
                "res": "f32" if io == "f32" or rng.random() < 0.5 else "bf16", "gate": rng.random() < 0.5,
                "post": rng.random() < 0.5, "scale": rng.random() < 0.5, "act": act}
    if op == "rotary":
        Hk, d = rng.randint(1, 8), rng.choice([64, 80, 128, 256])
        Hq = Hk * rng.randint(1, 8)
        train = rng.random() < 0.5
        case = {"op": op, "train": train, "T": _log(rng, 1, min(32768, (1 << 25) // ((Hq + Hk) * d))), "Hq": Hq, "Hk": Hk,
                "d": d, "rot": rng.choice([d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]), "inter": rng.random() < 0.5,
                "far": _log(rng, 1, 1000000), "factor": rng.choice([1.0, 4.0, 8.0]), "io": io}
        if not train:
            case["page"] = rng.choice([16, 64, 256])
        return case
    if op == "step_tables":
        R = _log(rng, 1, 4096)
        return {"op": op, "R": R, "held": rng.choice([0, _log(rng, 1, 8192)]), "new": _log(rng, 1, min(2047, 700000 // R)),
                "ragged": rng.random() < 0.5, "page": rng.choice([1, 16, 64, 256])}
    d, Hk, G, B = rng.choice([64, 128, 256]), rng.randint(1, 8), rng.randint(1, 8), rng.randint(1, 16)
    prefix = rng.choice([0, _log(rng, 1, 16384)])
    held = _log(rng, 1, 4096)
    # at most a fifth of the largest listed case's products, and 2 GiB of cache rows in fp32
    most = (1 << 34) // (5 * B * Hk * G * d * (prefix + held))
    R = _log(rng, 1, max(1, min(256, most, (1 << 28) // (Hk * d * held))))
    return {"op": op, "R": R, "B": B, "Hk": Hk, "G": G, "d": d, "prefix": prefix, "own": held,
            "page": rng.choice([16, 32, 64, 128]), "causal": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io = _TYPES[case.get("io", "bf16")]

    def randn(*shape, dtype=io, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def ints(lo, hi, *shape):  # lo .. hi inclusive
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int32)

    s = {"case": case}
    if case["op"] == "gated_norm":
        T, H, d = case["T"], case["H"], case["d"]
        s["x"] = randn(T, H, d)
        # the gate is the second half of one fused projection's rows
        s["gate"] = randn(T, 2 * H * d)[:, H * d:].unflatten(1, (H, d)) if case["gate"] else None
        s["weight"] = 1.0 + randn(d, dtype=torch.float32, scale=0.1)
        s["dy"] = randn(T, H, d) if case["train"] else None
    elif case["op"] == "residual_norm":
        T, C, res = case["T"], case["C"], _TYPES[case["res"]]
        s["x"] = randn(T, C, scale=0.5)
        s["residual"] = randn(T, C, dtype=res, scale=2.0)
        s["gate"] = randn(T, C) if case["gate"] else None
        s["w_pre"] = 1.0 + randn(C, dtype=torch.float32, scale=0.1)
        s["w_post"] = 1.0 + randn(C, dtype=torch.float32, scale=0.1) if case["post"] else None
        s["scale"] = 0.5 + randn(C, dtype=torch.float32, scale=0.1) if case["scale"] else None
        s["dy"] = randn(T, C) if case["train"] else None
        s["dh"] = randn(T, C, dtype=res) if case["train"] else None
    elif case["op"] == "rotary":
        T, Hq, Hk, d, half = case["T"], case["Hq"], case["Hk"], case["d"], case["rot"] // 2
        rows = randn(T, (Hq + 2 * Hk) * d)  # q, k, v of one fused projection
        s["q"], s["k"] = rows[:, :Hq * d].unflatten(1, (Hq, d)), rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
        s["v"] = rows[:, (Hq + Hk) * d:].unflatten(1, (Hk, d))
        s["positions"] = ints(0, case["far"], T)
        # base 10000, positions divided by the factor; attention scaled with it
        s["freqs"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half) / case["factor"]
        s["mscale"] = 1.0 + 0.1 * math.log(case["factor"])
        if case["train"]:
            s["dq"], s["dk"] = randn(T, Hq, d), randn(T, Hk, d)
        else:
            page = case["page"]
            pages = -(-T // page) + 2
            slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T]
            slots[16::17] = -1  # padded rows write nothing
            s["slots"] = slots
            s["k_cache"], s["v_cache"] = randn(pages, Hk, page, d), randn(pages, Hk, page, d)
    elif case["op"] == "step_tables":
        R, page = case["R"], case["page"]
        held = ints(0, case["held"], R)
        new = ints(0, case["new"], R) if case["ragged"] else torch.full((R,), case["new"], dtype=torch.int32, device="cuda")
        wide = -(-(case["held"] + case["new"]) // page)
        total = R * wide
        ids = torch.randperm(total + 7, generator=gen, device="cuda").to(torch.int32)
        s["seq_lens"], s["new_lens"] = held, new
        s["block_table"] = ids[:total].reshape(R, wide).clone()
        s["free_pages"] = ids.flip(0).contiguous()
        s["pages_used"] = torch.full((1,), 5, dtype=torch.int32, device="cuda")
        s["free_pages"] = torch.cat([s["free_pages"], ids[:5]])
        s["max_tokens"] = R * case["new"] + 3  # the buffers' capacity; rows behind the last token are padding
    else:
        R, B, Hk, G, d, page = case["R"], case["B"], case["Hk"], case["G"], case["d"], case["page"]
        held, prefix = case["own"], case["prefix"]
        wide, shared = -(-held // page), -(-prefix // page)
        pages = R * wide + shared
        ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["q"] = randn(R, B, Hk * G, d)
        s["k_cache"] = randn(pages, Hk, page, d, dtype=torch.bfloat16)
        s["v_cache"] = randn(pages, Hk, page, d, dtype=torch.bfloat16)
        s["prefix_table"] = ids[:shared].contiguous()
        s["block_table"] = ids[shared:].reshape(R, wide).contiguous()
        # ragged: the first request holds the whole length, the others from its half to the whole
        lens = ints((held + 1) // 2, held, R)
        lens[0] = held
        s["seq_lens"] = lens
    return s


# ---------------------------------------------------------------- the plain forms

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _act(g, act):
    """The gate's activation and its derivative."""
    if act == LINEAR:
        return g, torch.ones_like(g)
    p = torch.sigmoid(g)
    if act == SIGMOID:
        return p, p * (1 - p)
    return g * p, p * (1 + g * (1 - p))


EPS = 1e-6


def _plain_gated_norm(s):
    case, x = s["case"], s["x"].float()
    w = s["weight"]
    a, da = _act(s["gate"].float(), case["act"]) if case["gate"] else (1.0, None)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    io = s["x"].dtype
    out = {"y": (n * w * a).to(io)}
    if case["train"]:
        dy = s["dy"].float()
        dn = dy * w * a
        out["dx"] = (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(io)
        out["dweight"] = (dy * n * a).sum((0, 1))
        if case["gate"]:
            out["dgate"] = (dy * n * w * da).to(io)
    return out


def _plain_residual_norm(s):
    case, x, res = s["case"], s["x"].float(), s["residual"].float()
    io, rt = s["x"].dtype, s["residual"].dtype
    a, da = _act(s["gate"].float(), case["act"]) if case["gate"] else (1.0, None)
    sc = s["scale"] if case["scale"] else 1.0
    if case["post"]:
        r1 = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r1
        z = n * s["w_post"]
    else:
        z = x
    h = res + sc * a * z
    r2 = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    u = h * r2
    out = {"h": h.to(rt), "y": (u * s["w_pre"]).to(io)}
    if case["train"]:
        dy, dh = s["dy"].float(), s["dh"].float()
        du = dy * s["w_pre"]
        dh = dh + r2 * (du - u * (du * u).mean(-1, keepdim=True))
        out["dresidual"] = dh.to(rt)
        out["dw_pre"] = (dy * u).sum(0)
        if case["gate"]:
            out["dgate"] = (dh * sc * z * da).to(io)
        if case["scale"]:
            out["dscale"] = (dh * a * z).sum(0)
        dz = dh * sc * a
        if case["post"]:
            out["dw_post"] = (dz * n).sum(0)
            dn = dz * s["w_post"]
            dz = r1 * (dn - n * (dn * n).mean(-1, keepdim=True))
        out["dx"] = dz.to(io)
    return out


def _rotate(x, positions, freqs, mscale, inter, sign):
    # angles of far positions need 64 bits
    angle = positions.double()[:, None] * freqs[None]
    c, t = (torch.cos(angle) * mscale).float()[:, None], (torch.sin(angle) * (mscale * sign)).float()[:, None]
    half = freqs.numel()
    y = x.float()
    head, rest = y[..., :2 * half], y[..., 2 * half:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * c - b * t, a * t + b * c], -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat([a * c - b * t, a * t + b * c], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


def _plain_rotary(s):
    case = s["case"]
    rot = lambda x, sign: _rotate(x, s["positions"], s["freqs"], s["mscale"], case["inter"], sign)  # noqa: E731
    q, k = rot(s["q"], 1.0), rot(s["k"], 1.0)
    if case["train"]:
        return {"q": q, "k": k, "dq": rot(s["dq"], -1.0), "dk": rot(s["dk"], -1.0)}
    page, slots = case["page"], s["slots"]
    live = slots >= 0
    at, off = slots[live] // page, slots[live] % page
    s["k_cache"][at, :, off] = k[live]
    s["v_cache"][at, :, off] = s["v"][live]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_step_tables(s):
    page, held, new = s["case"]["page"], s["seq_lens"].long(), s["new_lens"].long()
    R, M = held.numel(), s["max_tokens"]
    cu = torch.zeros(R + 1, dtype=torch.int64, device=held.device)
    cu[1:] = torch.cumsum(new, 0)
    have, need = (held + page - 1) // page, (held + new + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have)
    used = s["pages_used"].long()
    column = torch.arange(s["block_table"].shape[1], device=held.device)[None]
    fresh = (column >= have[:, None]) & (column < need[:, None])
    at = (used + first[:, None] + column - have[:, None]).clamp(0, s["free_pages"].numel() - 1)
    table = torch.where(fresh, s["free_pages"][at], s["block_table"])
    token = torch.arange(M, device=held.device)
    row = torch.searchsorted(cu[1:].contiguous(), token, right=True).clamp(max=R - 1)
    live = token < cu[-1]
    pos = torch.where(live, held[row] + token - cu[row], 0)
    slot = torch.where(live, table[row, pos // page].long() * page + pos % page, -1)
    s["block_table"].copy_(table)
    return {"cu_new": cu.int(), "positions": pos.int(), "slots": slot, "seq_lens": (held + new).int(),
            "pages_used": (used + (need - have).sum()).int(), "block_table": s["block_table"],
            "status": torch.zeros(1, dtype=torch.int32, device=held.device)}


def _plain_attention(s):
    case = s["case"]
    R, B, Hk, G, d, prefix = case["R"], case["B"], case["Hk"], case["G"], case["d"], case["prefix"]
    q = s["q"].float().reshape(R, B, Hk, G, d) / math.sqrt(d)
    lens = s["seq_lens"].long()
    # the requests' own keys [R, Hk, L, d], rows behind a request's length cleared
    L = s["block_table"].shape[1] * case["page"]
    seen = torch.arange(L, device=q.device)[None] < lens[:, None]
    ko, vo = (torch.where(seen[:, None, :, None], c[s["block_table"].long()].transpose(1, 2).reshape(R, Hk, L, d), 0).float()
              for c in (s["k_cache"], s["v_cache"]))
    qo = q.permute(0, 2, 1, 3, 4).reshape(R, Hk, B * G, d)
    so = torch.matmul(qo, ko.transpose(2, 3).contiguous())
    last = lens[:, None] - (B - 1 - torch.arange(B, device=q.device))[None] if case["causal"] else lens[:, None].expand(R, B)
    open_ = torch.arange(L, device=q.device) < last.repeat_interleave(G, 1)[:, None, :, None]
    so = so.masked_fill(~open_, -math.inf)
    # the shared prefix [Hk, prefix, d] against every request's rows
    kp, vp = (c[s["prefix_table"].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :prefix].float()
              for c in (s["k_cache"], s["v_cache"]))
    qp = q.permute(2, 0, 1, 3, 4).reshape(Hk, R * B * G, d)
    sp = torch.matmul(qp, kp.transpose(1, 2).contiguous())
    top = so.amax(-1)
    if prefix:
        top = torch.maximum(top, sp.amax(-1).reshape(Hk, R, B * G).transpose(0, 1))
    base = top.masked_fill(top == -math.inf, 0.0)
    po = torch.exp(so - base[..., None])
    pp = torch.exp(sp - base.transpose(0, 1).reshape(Hk, R * B * G)[..., None])
    total = po.sum(-1) + pp.sum(-1).reshape(Hk, R, B * G).transpose(0, 1)
    o = torch.matmul(po, vo) + torch.matmul(pp, vp).reshape(Hk, R, B * G, d).transpose(0, 1)
    o = o / total.clamp(min=1e-38)[..., None]
    lse = torch.log(total) + base
    o = o.reshape(R, Hk, B, G, d).transpose(1, 2).reshape(R, B, Hk * G, d)
    return {"o": o.to(s["q"].dtype), "lse": lse.reshape(R, Hk, B, G).transpose(1, 2).reshape(R, B, Hk * G)}


_PLAIN = {"gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm, "rotary": _plain_rotary,
          "step_tables": _plain_step_tables, "attention": _plain_attention}


# ---------------------------------------------------------------- the library's calls

def _own_gated_norm(s):
    import gated_deltanet_dual_amd as g
    case = s["case"]
    if not case["train"]:
        return {"y": g.gated_norm(s["x"], s["weight"], s["gate"], activation=case["act"], eps=EPS)}
    y, rstd = g.gated_norm(s["x"], s["weight"], s["gate"], activation=case["act"], eps=EPS, want_rstd=True)
    dx, dgate, dweight = g.gated_norm_bwd(s["x"], s["weight"], s["gate"], s["dy"], rstd, activation=case["act"])
    out = {"y": y, "dx": dx, "dweight": dweight}
    if case["gate"]:
        out["dgate"] = dgate
    return out


def _own_residual_norm(s):
    import gated_deltanet_dual_amd as g
    case = s["case"]
    args = (s["x"], s["residual"], s["w_pre"])
    more = dict(w_post=s["w_post"], gate=s["gate"], scale=s["scale"], activation=case["act"])
    if not case["train"]:
        h, y = g.residual_norm(*args, **more, eps=EPS)
        return {"h": h, "y": y}
    h, y, rstd = g.residual_norm(*args, **more, eps=EPS, want_rstd=True)
    grads = g.residual_norm_bwd(*args, s["dy"], s["dh"], rstd, **more)
    return {"h": h, "y": y, **{name: t for name, t in grads.items() if t is not None}}


def _own_rotary(s):
    import gated_deltanet_dual_amd as g
    case = s["case"]
    more = dict(interleaved=case["inter"], mscale=s["mscale"])
    if case["train"]:
        q, k = g.rotary(s["positions"], s["freqs"], s["q"], s["k"], **more)
        dq, dk = g.rotary(s["positions"], s["freqs"], s["dq"], s["dk"], inverse=True, **more)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    q = g.rotary_cache(s["positions"], s["freqs"], s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], **more)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_step_tables(s):
    import gated_deltanet_dual_amd as g
    t = g.step_tables(s["seq_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["pages_used"],
                      s["case"]["page"], s["max_tokens"])
    return {**t, "block_table": s["block_table"]}


def _own_attention(s):
    import gated_deltanet_dual_amd as g
    case = s["case"]
    o, lse = g.block_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                               prefix_table=s["prefix_table"], prefix_len=case["prefix"], causal=case["causal"],
                               want_lse=True)
    return {"o": o, "lse": lse}


_OWN = {"gated_norm": _own_gated_norm, "residual_norm": _own_residual_norm, "rotary": _own_rotary,
        "step_tables": _own_step_tables, "attention": _own_attention}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case.get("io", "bf16") == "bf16" else 4
    if case["op"] == "gated_norm":
        n, gate = case["T"] * case["H"] * case["d"], 1 if case["gate"] else 0
        # forward reads x and the gate and writes y; the reverse mode reads dy (x and the gate are the same
        # inputs, counted once) and writes dx and the gate's gradient
        tensors = 2 + gate + (2 + gate if case["train"] else 0)
        return {"bytes": tensors * n * e + 4 * case["d"] * (1 + case["train"]), "flops": n * (6 + 14 * case["train"])}
    if case["op"] == "residual_norm":
        n, gate, r = case["T"] * case["C"], 1 if case["gate"] else 0, 2 if case["res"] == "bf16" else 4
        io, res = 2 + gate, 2
        if case["train"]:
            io, res = io + 2 + gate, res + 2
        weights = 1 + case["post"] + case["scale"]
        return {"bytes": n * (io * e + res * r) + 4 * case["C"] * weights * (1 + case["train"]),
                "flops": n * (10 + 24 * case["train"])}
    if case["op"] == "rotary":
        T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
        heads = 2 * (Hq + Hk) * (2 if case["train"] else 1) + (0 if case["train"] else 2 * Hk)
        return {"bytes": T * (heads * d * e + 4 + (0 if case["train"] else 8)) + 4 * case["rot"],
                "flops": T * (Hq + Hk) * case["rot"] * 3 * (2 if case["train"] else 1)}
    if case["op"] == "step_tables":
        tokens = case["R"] * case["new"] * (0.5 if case["ragged"] else 1.0)
        # lengths in and out, the offsets, one table entry and one free page for each new page, and 12 bytes a row
        return {"bytes": 16 * case["R"] + 8 * (tokens / case["page"] + case["R"]) + 12 * (case["R"] * case["new"] + 3),
                "flops": 4 * tokens}
    R, rows, Hk, d = case["R"], case["B"] * case["G"], case["Hk"], case["d"]
    kept = case["own"] * (0.75 if R > 1 else 1.0)  # the mean length
    return {"bytes": 4 * Hk * d * (case["prefix"] + R * kept) + R * rows * Hk * (4 * d + 4)
            + 4 * (R + (case["prefix"] + R * kept) / case["page"]),
            "flops": 4 * d * R * rows * Hk * (case["prefix"] + kept)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "step_tables":
        return None  # whole numbers
    return _EXACT[case["op"]](prepare(case, seed))


def _gate64(s, leaf):
    act = s["case"]["act"]
    return leaf if act == LINEAR else torch.sigmoid(leaf) if act == SIGMOID else leaf / (1 + torch.exp(-leaf))


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _rms64(x, w):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def _exact_gated_norm(s):
    x, w, g = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["gate"])
    y = _rms64(x, w)
    if g is not None:
        y = y * _gate64(s, g)
    out = {"y": y.detach()}
    if s["dy"] is not None:
        y.backward(s["dy"].double())
        out |= {"dx": x.grad, "dweight": w.grad}
        if g is not None:
            out["dgate"] = g.grad
    return out


def _exact_residual_norm(s):
    x, res, g, w2, w1, sc = (_leaf(s[n]) for n in ("x", "residual", "gate", "w_pre", "w_post", "scale"))
    z = x if w1 is None else _rms64(x, w1)
    if g is not None:
        z = z * _gate64(s, g)
    if sc is not None:
        z = z * sc
    h = res + z
    y = _rms64(h, w2)
    out = {"h": h.detach(), "y": y.detach()}
    if s["dy"] is not None:
        torch.autograd.backward([h, y], [s["dh"].double(), s["dy"].double()])
        out |= {n: t.grad for n, t in (("dx", x), ("dresidual", res), ("dgate", g), ("dw_pre", w2), ("dw_post", w1),
                                       ("dscale", sc)) if t is not None}
    return out


def _turn64(s, x, sign):
    """The rotation as a product of complex numbers."""
    n = s["freqs"].numel()
    y = x.double().clone()
    i = torch.arange(n, device=x.device)
    re, im = (2 * i, 2 * i + 1) if s["case"]["inter"] else (i, n + i)
    unit = torch.polar(torch.full_like(s["freqs"], s["mscale"])[None].expand(x.shape[0], n).contiguous(),
                       sign * s["positions"].double()[:, None] * s["freqs"])
    turned = torch.complex(y[..., re], y[..., im]) * unit[:, None]
    y[..., re], y[..., im] = turned.real, turned.imag
    return y


def _exact_rotary(s):
    q, k = _turn64(s, s["q"], 1.0), _turn64(s, s["k"], 1.0)
    if s["case"]["train"]:
        return {"q": q, "k": k, "dq": _turn64(s, s["dq"], -1.0), "dk": _turn64(s, s["dk"], -1.0)}
    kc, vc, page = s["k_cache"].double(), s["v_cache"].double(), s["case"]["page"]
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    where = s["slots"][rows]
    kc.transpose(1, 2)[where // page, where % page] = k[rows]
    vc.transpose(1, 2)[where // page, where % page] = s["v"][rows].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    case = s["case"]
    R, B, Hk, G, d, prefix, page = (case[n] for n in ("R", "B", "Hk", "G", "d", "prefix", "page"))
    o = torch.zeros(R, B, Hk * G, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((R, B, Hk * G), -math.inf, dtype=torch.float64, device=s["q"].device)

    def rows(cache, table, n):  # [Hk, n, d]
        pages = cache[table[:-(-n // page)].long()].double()
        return pages.permute(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n]

    kp, vp = rows(s["k_cache"], s["prefix_table"], prefix), rows(s["v_cache"], s["prefix_table"], prefix)
    for r, n in enumerate(s["seq_lens"].tolist()):
        k = torch.cat([kp, rows(s["k_cache"], s["block_table"][r], n)], 1)
        v = torch.cat([vp, rows(s["v_cache"], s["block_table"][r], n)], 1)
        for b in range(B) if case["causal"] else [slice(None)]:
            m = prefix + (max(0, n - (B - 1 - b)) if case["causal"] else n)
            if m == 0:
                continue
            q = s["q"][r, b].double().reshape(-1, Hk, G, d).permute(1, 0, 2, 3).reshape(Hk, -1, d)
            z = torch.matmul(q, k[:, :m].transpose(1, 2).contiguous()) * d ** -0.5
            o[r, b] = torch.matmul(torch.softmax(z, -1), v[:, :m]).reshape(Hk, -1, G, d).transpose(0, 1).reshape(-1, Hk * G, d).reshape(o[r, b].shape)
            lse[r, b] = torch.logsumexp(z, -1).reshape(Hk, -1, G).transpose(0, 1).reshape(lse[r, b].shape)
    return {"o": o, "lse": lse}


_EXACT = {"gated_norm": _exact_gated_norm, "residual_norm": _exact_residual_norm, "rotary": _exact_rotary,
          "attention": _exact_attention}
