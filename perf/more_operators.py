"""What the softmax layers of a hybrid model do with their queries, keys and values, as cases to measure: the norms of
queries and keys for each head with the position rotation in the same pass, both directions; the same on the way into
a paged cache, in the tensors' own type or in 4 bits; rows read back from a cache in 4 bits; and the block attention
over such a cache.

A cache in 4 bits holds a row's channels in groups of 32, each value one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign,
times the group's power of two.

Each case is one call, or a forward with its reverse mode, or rows written and all rows read, as a user's program makes
it.  `run` computes the plain form with elementary torch operations or, where `own` is set, calls the library.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one request: only latency counts
        {"name": "qk_norm_rotary_token", "op": "qk_norm_rotary", "train": False, "T": 1, "Hk": 4, "G": 4, "d": 128, "rot": 128,
         "inter": False, "far": 8192, "factor": 1.0, "io": "bf16", "norm": "qk"},
        # the training step of 4 x 8192 tokens, q and k slices of one projection, forward and reverse mode
        {"name": "qk_norm_rotary_train", "op": "qk_norm_rotary", "train": True, "T": 32768, "Hk": 4, "G": 4, "d": 128, "rot": 128,
         "inter": False, "far": 8192, "factor": 1.0, "io": "bf16", "norm": "qk"},
        # an fp32 run with odd head counts, a head width that is no power of two and 50 of its channels turned
        {"name": "qk_norm_rotary_fp32_odd", "op": "qk_norm_rotary", "train": True, "T": 1531, "Hk": 3, "G": 2, "d": 80, "rot": 50,
         "inter": True, "far": 4096, "factor": 1.0, "io": "f32", "norm": "qk"},
        # the serving step of 256 requests x 4 tokens into a cache of the tensors' own type, a quarter of each head turned
        {"name": "cache_step_bf16", "op": "cache", "bits": 16, "T": 1024, "Hk": 4, "G": 4, "d": 128, "rot": 32, "inter": False,
         "far": 8192, "factor": 1.0, "io": "bf16", "norm": "qk", "page": 64},
        # the same step into a cache in 4 bits
        {"name": "cache_step_fp4", "op": "cache", "bits": 4, "T": 1024, "Hk": 4, "G": 4, "d": 128, "rot": 128, "inter": False,
         "far": 8192, "factor": 1.0, "io": "bf16", "norm": "qk", "page": 64},
        # prompts of 16384 tokens in all into the cache in 4 bits, far into a scaled context
        {"name": "cache_prompt_fp4", "op": "cache", "bits": 4, "T": 16384, "Hk": 4, "G": 4, "d": 128, "rot": 128, "inter": True,
         "far": 1000000, "factor": 8.0, "io": "bf16", "norm": "qk", "page": 64},
        # one request, one token, a short cache of small pages: only latency counts
        {"name": "attention_fp4_token", "op": "attention", "R": 1, "B": 1, "Hk": 4, "G": 4, "d": 128, "prefix": 0, "own": 257,
         "page": 16, "causal": False},
        # one request, one token, a long cache of its own
        {"name": "attention_fp4_token_long", "op": "attention", "R": 1, "B": 1, "Hk": 4, "G": 4, "d": 128, "prefix": 0,
         "own": 131072, "page": 64, "causal": False},
        # 256 requests x 4 tokens over up to 1024 tokens each of their own
        {"name": "attention_fp4_step", "op": "attention", "R": 256, "B": 4, "Hk": 4, "G": 4, "d": 128, "prefix": 0, "own": 1024,
         "page": 64, "causal": False},
        # the same requests over a shared prefix of 8192 tokens as well
        {"name": "attention_fp4_shared_prefix", "op": "attention", "R": 256, "B": 4, "Hk": 4, "G": 4, "d": 128, "prefix": 8192,
         "own": 1024, "page": 64, "causal": False},
        # a draft of 7 tokens verified causally: 37 requests, odd prefix, small pages, wide heads
        {"name": "attention_fp4_verify_odd", "op": "attention", "R": 37, "B": 7, "Hk": 2, "G": 8, "d": 256, "prefix": 2500,
         "own": 777, "page": 16, "causal": True},
        # narrow heads, each with its own keys, a short prefix
        {"name": "attention_fp4_narrow", "op": "attention", "R": 61, "B": 5, "Hk": 8, "G": 1, "d": 64, "prefix": 300, "own": 3000,
         "page": 32, "causal": True},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rotary", "cache", "attention"])
    Hk, G = rng.randint(1, 8), rng.randint(1, 8)
    if op != "attention":
        bits = rng.choice([4, 4, 16])
        if op == "cache" and bits == 4:
            d = rng.choice([32, 64, 96, 128, 128, 160, 256])
        else:
            d = rng.choice([64, 80, 128, 128, 256, rng.randint(2, 300)])
        case = {"op": op, "T": _log(rng, 1, min(32768, (1 << 26) // (Hk * (G + 2) * d))), "Hk": Hk, "G": G, "d": d,
                "rot": rng.choice([d // 2 * 2, d // 4 * 2, 2 * rng.randint(0, d // 2)]), "inter": rng.random() < 0.5,
                "far": _log(rng, 1, 1000000), "factor": rng.choice([1.0, 4.0, 8.0]), "io": rng.choice(["bf16", "bf16", "f32"]),
                "norm": rng.choice(["qk", "qk", "qk", "k", "q"])}
        if op == "cache":
            return {**case, "bits": bits, "page": rng.choice([1, 16, 64, 256])}
        return {**case, "train": rng.random() < 0.6}
    d, B = rng.choice([64, 128, 128, 256]), rng.randint(1, 16)
    prefix = rng.choice([0, _log(rng, 1, 16384)])
    held = _log(rng, 1, 65536)
    # at most a fifth of the largest listed case's products, and 2 GiB of cache rows in fp32
    most = (1 << 34) // (5 * B * Hk * G * d * (prefix + held))
    R = _log(rng, 1, max(1, min(256, most, (1 << 28) // (Hk * d * held))))
    return {"op": op, "R": R, "B": B, "Hk": Hk, "G": G, "d": d, "prefix": prefix, "own": held,
            "page": rng.choice([16, 32, 64, 128]), "causal": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io = _TYPES[case.get("io", "bf16")]

    def randn(*shape, dtype=io, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    def ints(lo, hi, *shape):  # lo .. hi inclusive
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int32)

    def cache4(pages, heads, page, d):  # (codes, scales) of rows that are normal
        codes, scales = _to_4_bits(randn(pages, heads, page, d, dtype=torch.float32))
        return codes, scales.transpose(2, 3).contiguous()

    s = {"case": case}
    if case["op"] == "attention":
        R, B, Hk, G, d, page = case["R"], case["B"], case["Hk"], case["G"], case["d"], case["page"]
        held, prefix = case["own"], case["prefix"]
        wide, shared = -(-held // page), -(-prefix // page)
        pages = R * wide + shared
        ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        s["q"] = randn(R, B, Hk * G, d)
        s["k_cache"], s["v_cache"] = cache4(pages, Hk, page, d), cache4(pages, Hk, page, d)
        s["prefix_table"] = ids[:shared].contiguous()
        s["block_table"] = ids[shared:].reshape(R, wide).contiguous()
        # ragged: the first request holds the whole length, the others from its half to the whole
        lens = ints((held + 1) // 2, held, R)
        lens[0] = held
        s["seq_lens"] = lens
        return s
    T, Hk, Hq, d, half = case["T"], case["Hk"], case["Hk"] * case["G"], case["d"], case["rot"] // 2
    rows = randn(T, (Hq + 2 * Hk) * d)  # q, k, v of one fused projection
    s["q"], s["k"] = rows[:, :Hq * d].unflatten(1, (Hq, d)), rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    s["v"] = rows[:, (Hq + Hk) * d:].unflatten(1, (Hk, d))
    s["positions"] = ints(0, case["far"], T)
    # base 10000, positions divided by the factor; attention scaled with it
    s["freqs"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1)) / case["factor"]
    s["mscale"] = 1.0 + 0.1 * math.log(case["factor"])
    # weights of the norms; a side without one is turned but not normed
    s["q_weight"] = 1.0 + randn(d, dtype=torch.float32, scale=0.1) if "q" in case["norm"] else None
    s["k_weight"] = 1.0 + randn(d, dtype=torch.float32, scale=0.1) if "k" in case["norm"] else None
    if case["op"] == "qk_norm_rotary":
        if case["train"]:
            s["dq"], s["dk"] = randn(T, Hq, d), randn(T, Hk, d)
        return s
    page = case["page"]
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T]
    slots[16::17] = -1  # padded rows write nothing
    s["slots"] = slots
    if case["bits"] == 4:
        s["k_cache"], s["v_cache"] = cache4(pages, Hk, page, d), cache4(pages, Hk, page, d)
        s["all_slots"] = torch.arange(pages * page, device="cuda")
    else:
        s["k_cache"], s["v_cache"] = randn(pages, Hk, page, d), randn(pages, Hk, page, d)
    return s


# ---------------------------------------------------------------- the plain forms

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _to_4_bits(x):
    """x [..., d] as (codes uint8 [..., d / 2], scales uint8 [..., d / 32]): the lower four bits of a byte are the even
    channel's.  A group's exponent is that of its largest value less two, and one more where that value is above 7
    units, so that none is cut by more than half a step; the byte is the exponent + 127, 255 for a group with an
    infinity or NaN."""
    x = x.unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    e = torch.frexp(torch.where(fine, top, 1.0))[1].long() - 3
    one = torch.ones((), dtype=torch.float64, device=x.device)
    e = (e + (torch.where(fine, top, 1.0) > 7 * torch.ldexp(one, e))).clamp(-126, 125)
    m = (x.abs() * torch.ldexp(one, -e)[..., None]).nan_to_num()
    # halfway goes to the even code
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = (code + 8 * (x < 0)).to(torch.uint8).flatten(-2)
    scales = torch.where(fine, e + 127, 255).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], scales


def _from_4_bits(codes, scales):
    """The fp32 values [..., d] of codes [..., d / 2] and scales [..., d / 32]."""
    dev = codes.device
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=dev)
    value = torch.cat([value, -value])
    pair = torch.stack([value.repeat(16), value.repeat_interleave(16)], -1)  # of a byte's two codes
    scale = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan], device=dev)
    x = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32)) * scale[scales.int()][..., None]
    return x.flatten(-2)


def _turn(x, s, sign):
    """x [T, H, d] fp32 or fp64, its first channels turned by the positions."""
    # angles of far positions need 64 bits
    angle = s["positions"].double()[:, None] * s["freqs"][None]
    c = (torch.cos(angle) * s["mscale"]).to(x.dtype)[:, None]
    t = (torch.sin(angle) * (s["mscale"] * sign)).to(x.dtype)[:, None]
    half = s["freqs"].numel()
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if s["case"]["inter"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * c - b * t, a * t + b * c], -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat([a * c - b * t, a * t + b * c], -1)
    return torch.cat([turned, rest], -1)


def _norm_turn(x, w, s, dtype=torch.float32):
    x = x.to(dtype)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(dtype)
    return _turn(x, s, 1.0)


def _plain_reverse(x, w, dy, s):
    """(dx, dw) of _norm_turn."""
    io, x = x.dtype, x.float()
    du = _turn(dy.float(), s, -1.0)
    if w is None:
        return du.to(io), None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    dn = du * w
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(io), (du * n).sum((0, 1))


def _plain_qk_norm_rotary(s):
    io = s["q"].dtype
    out = {"q": _norm_turn(s["q"], s["q_weight"], s).to(io), "k": _norm_turn(s["k"], s["k_weight"], s).to(io)}
    if s["case"]["train"]:
        out["dq"], out["dq_weight"] = _plain_reverse(s["q"], s["q_weight"], s["dq"], s)
        out["dk"], out["dk_weight"] = _plain_reverse(s["k"], s["k_weight"], s["dk"], s)
    return out


def _plain_cache(s):
    case, io, slots = s["case"], s["q"].dtype, s["slots"]
    page = case["page"]
    live = slots >= 0
    at, off = slots[live] // page, slots[live] % page
    out = {"q": _norm_turn(s["q"], s["q_weight"], s).to(io)}
    if case["bits"] == 16:
        s["k_cache"][at, :, off] = _norm_turn(s["k"], s["k_weight"], s).to(io)[live]
        s["v_cache"][at, :, off] = s["v"][live]
        return {**out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    # values next to the border of two codes need 64 bits
    for name, x in (("k", _norm_turn(s["k"], s["k_weight"], s, torch.float64)), ("v", s["v"].double())):
        codes, scales = s[name + "_cache"]
        c, e = _to_4_bits(x[live])
        codes[at, :, off] = c
        scales[at, :, :, off] = e
        at_all, off_all = s["all_slots"] // page, s["all_slots"] % page
        out[name] = _from_4_bits(codes[at_all, :, off_all], scales[at_all, :, :, off_all]).to(io)
    return out


def _plain_attention(s):
    case = s["case"]
    R, B, Hk, G, d, prefix = case["R"], case["B"], case["Hk"], case["G"], case["d"], case["prefix"]
    q = s["q"].float().reshape(R, B, Hk, G, d) / math.sqrt(d)
    lens = s["seq_lens"].long()

    def rows(cache, table):  # the pages' rows, fp32 [..., pages, Hk, page, d]
        codes, scales = cache
        return _from_4_bits(codes[table.long()], scales[table.long()].transpose(-1, -2))

    # the requests' own keys [R, Hk, L, d], rows behind a request's length cleared
    L = s["block_table"].shape[1] * case["page"]
    seen = torch.arange(L, device=q.device)[None] < lens[:, None]
    ko, vo = (torch.where(seen[:, None, :, None], rows(c, s["block_table"]).transpose(1, 2).reshape(R, Hk, L, d), 0)
              for c in (s["k_cache"], s["v_cache"]))
    qo = q.permute(0, 2, 1, 3, 4).reshape(R, Hk, B * G, d)
    so = torch.matmul(qo, ko.transpose(2, 3).contiguous())
    last = lens[:, None] - (B - 1 - torch.arange(B, device=q.device))[None] if case["causal"] else lens[:, None].expand(R, B)
    open_ = torch.arange(L, device=q.device) < last.repeat_interleave(G, 1)[:, None, :, None]
    so = so.masked_fill(~open_, -math.inf)
    # the shared prefix [Hk, prefix, d] against every request's rows
    kp, vp = (rows(c, s["prefix_table"]).transpose(0, 1).reshape(Hk, -1, d)[:, :prefix] for c in (s["k_cache"], s["v_cache"]))
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


_PLAIN = {"qk_norm_rotary": _plain_qk_norm_rotary, "cache": _plain_cache, "attention": _plain_attention}


# ---------------------------------------------------------------- the library's calls

def _own_qk_norm_rotary(s):
    import gated_deltanet_dual_amd as g
    args = (s["positions"], s["freqs"], s["q"], s["k"])
    more = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["case"]["inter"], mscale=s["mscale"])
    q, k = g.qk_norm_rotary(*args, **more)
    out = {"q": q, "k": k}
    if s["case"]["train"]:
        out |= g.qk_norm_rotary_bwd(*args, s["dq"], s["dk"], **more)
    return out


def _own_cache(s):
    import gated_deltanet_dual_amd as g
    write = g.qk_norm_rotary_cache_fp4 if s["case"]["bits"] == 4 else g.qk_norm_rotary_cache
    q = write(s["positions"], s["freqs"], s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["case"]["inter"], mscale=s["mscale"])
    if s["case"]["bits"] == 16:
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    k, v = g.cache_fp4_rows(s["all_slots"], s["k_cache"], s["v_cache"], dtype=s["q"].dtype)
    return {"q": q, "k": k, "v": v}


def _own_attention(s):
    import gated_deltanet_dual_amd as g
    case = s["case"]
    o, lse = g.block_attention_fp4(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                   prefix_table=s["prefix_table"], prefix_len=case["prefix"], causal=case["causal"],
                                   want_lse=True)
    return {"o": o, "lse": lse}


_OWN = {"qk_norm_rotary": _own_qk_norm_rotary, "cache": _own_cache, "attention": _own_attention}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    Hk, G, d = case["Hk"], case["G"], case["d"]
    row4 = d / 2 + d / 32  # bytes of a row in 4 bits
    if case["op"] == "attention":
        R, B, page = case["R"], case["B"], case["page"]
        kept = case["own"] * (0.75 if R > 1 else 1.0)  # the mean length
        return {"bytes": 2 * Hk * row4 * (case["prefix"] + R * kept) + R * B * G * Hk * (4 * d + 4)
                + 4 * (R + (case["prefix"] + R * kept) / page),
                "flops": 4 * d * R * B * G * Hk * (case["prefix"] + kept)}
    e, T = 2 if case["io"] == "bf16" else 4, case["T"]
    turns = T * Hk * (G + 1) * case["rot"] * 3
    norms = T * Hk * d * 4 * (G * ("q" in case["norm"]) + ("k" in case["norm"]))
    if case["op"] == "qk_norm_rotary":
        # the reverse mode reads the outputs' gradients (q and k are the same inputs, counted once) and writes the inputs'
        tensors = 4 if case["train"] else 2
        return {"bytes": tensors * T * Hk * (G + 1) * d * e + T * 4 + 4 * case["rot"] + 4 * d * tensors,
                "flops": (turns + norms) * (3 if case["train"] else 1)}
    read = T * (Hk * (G + 2) * d * e + 4 + 8) + 4 * case["rot"] + 8 * d
    if case["bits"] == 16:
        return {"bytes": read + T * Hk * (G + 2) * d * e, "flops": turns + norms}
    # and all rows of the cache read back
    rows = (-(-T // case["page"]) + 2) * case["page"]
    return {"bytes": read + T * Hk * (G * d * e + 2 * row4) + rows * (8 + 2 * Hk * (row4 + d * e)),
            "flops": turns + norms + 4 * T * Hk * d + 2 * rows * Hk * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _defined(s, x, w):
    """The norm, then the rotation as a product of complex numbers."""
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    n = s["freqs"].numel()
    i = torch.arange(n, device=x.device)
    re, im = (2 * i, 2 * i + 1) if s["case"]["inter"] else (i, n + i)
    angle = s["positions"].double()[:, None] * s["freqs"]
    z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None]
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_qk_norm_rotary(s):
    out = {}
    for name in ("q", "k"):
        x, w = _leaf(s[name]), _leaf(s[name + "_weight"])
        y = _defined(s, x, w)
        out[name] = y.detach()
        if s["case"]["train"]:
            y.backward(s["d" + name].double())
            out["d" + name] = x.grad
            if w is not None:
                out["d%s_weight" % name] = w.grad
    return out


def _nearest(x):
    """x [..., d] as the values that 4 bits and a power of two for 32 of them hold."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = g.abs().max(-1, keepdim=True).values
    unit = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 2), torch.ones_like(top))
    unit = torch.where(top > 7 * unit, 2 * unit, unit).clamp(2.0 ** -126, 2.0 ** 125)
    z = g / unit
    # steps of 1/2 below 2, 1 below 4, 2 below 8; torch.round goes to the even one
    step = torch.where(z.abs() < 2, 0.5, torch.where(z.abs() < 4, 1.0, 2.0))
    return ((torch.round(z / step) * step).clamp(-6, 6) * unit).reshape(x.shape)


def _values(cache, rows=None):
    """The values of a cache's pages in 64 bits, [pages, heads, page, d]."""
    codes, scales = cache if rows is None else (cache[0][rows], cache[1][rows])
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    m, e = (c & 1).double(), ((c >> 1) & 3).double()
    size = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    unit = torch.exp2(scales.double() - 127).transpose(-1, -2).repeat_interleave(32, -1)
    return torch.where(c >= 8, -size, size) * unit


def _exact_cache(s):
    case, page = s["case"], s["case"]["page"]
    out = {"q": _defined(s, s["q"].double(), s["q_weight"])}
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    where = s["slots"][rows]
    for name, x in (("k", _defined(s, s["k"].double(), s["k_weight"])), ("v", s["v"].double())):
        cache = s[name + "_cache"]
        held = (_values(cache) if case["bits"] == 4 else cache.double()).transpose(1, 2)
        held[where // page, where % page] = (_nearest(x) if case["bits"] == 4 else x)[rows]
        if case["bits"] == 4:
            out[name] = held.flatten(0, 1)
        else:
            out[name + "_cache"] = held.transpose(1, 2)
    return out


def _exact_attention(s):
    case = s["case"]
    R, B, Hk, G, d, prefix, page = (case[n] for n in ("R", "B", "Hk", "G", "d", "prefix", "page"))
    o = torch.zeros(R, B, Hk * G, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((R, B, Hk * G), -math.inf, dtype=torch.float64, device=s["q"].device)

    def rows(cache, table, n):  # [Hk, n, d]
        pages = _values(cache, table[:-(-n // page)].long())
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


_EXACT = {"qk_norm_rotary": _exact_qk_norm_rotary, "cache": _exact_cache, "attention": _exact_attention}
