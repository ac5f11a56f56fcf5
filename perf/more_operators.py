"""Workloads of what stands around a softmax-attention layer when it has
positions and serves from pages.

  rope    ``qk_norm_rope_fwd``, and with ``grad`` also ``qk_norm_rope_bwd``: the
          norm of every query and key head and the rotation by position;
  append  ``kv_append``: new keys (rotated on the way) and values into pages,
          16-bit or fp32 ones, or 4-bit ones that are then read back;
  gather  ``kv_gather``: the rows' tokens out of their pages, as the prompt
          attention takes them;
  paged   ``attn_paged``: one or a few new tokens per row against the pages.

With ``own`` false the same values come from elementary torch operations in
fp32, rounded once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
GROUP = 32  # values that share a step in a 4-bit cache


# ------------------------------------------------------------------ cases

def _rope(name, lengths, H, Hkv, D, R, grad, dtype="bf16", batch=0, norm=True, interleaved=False,
          first=0, fused=False):
    """``lengths``: packed sequences as text "5,37" (positions given), or with
    batch > 0 that many rows of one length; first: their first position."""
    c = {"op": "rope", "lengths": lengths, "H": H, "Hkv": Hkv, "D": D, "R": R, "grad": grad,
         "dtype": dtype, "batch": batch, "norm": norm, "interleaved": interleaved, "first": first,
         "fused": fused}
    return dict(c, name=name) if name else c


def _append(name, lengths, used, H, Hkv, D, R, page, bits, dtype="bf16", interleaved=False,
            fused=False):
    """Row b appends ``lengths[b]`` tokens behind its first ``used[b]``; H > 0:
    queries of that many heads are rotated too."""
    c = {"op": "append", "lengths": lengths, "used": used, "H": H, "Hkv": Hkv, "D": D, "R": R,
         "page": page, "bits": bits, "dtype": dtype, "interleaved": interleaved, "fused": fused}
    return dict(c, name=name) if name else c


def _gather(name, lengths, Hkv, D, page, bits, dtype="bf16"):
    c = {"op": "gather", "lengths": lengths, "Hkv": Hkv, "D": D, "page": page, "bits": bits,
         "dtype": dtype}
    return dict(c, name=name) if name else c


def _paged(name, B, S, used, T, H, Hkv, D, page, bits, dtype="bf16"):
    """B rows of at most S tokens, spread over [used, 1] of S."""
    c = {"op": "paged", "B": B, "S": S, "used": used, "T": T, "H": H, "Hkv": Hkv, "D": D,
         "page": page, "bits": bits, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    ones = ",".join(["1"] * 64)
    fill = ",".join(str(300 + 1700 * i // 63) for i in range(64))
    return [
        # a decode step's queries and keys
        _rope("rope_decode", "1", 16, 4, 128, 128, False, batch=64, first=1500),
        # an attention layer in training, at the shape of the mixers' 300M workload
        _rope("rope_train", "2048", 8, 8, 128, 128, True, batch=16),
        # packed fine-tuning samples, q and k views of one projection, half of a head rotated
        _rope("rope_packed", "3001,700,129,4096,15,251", 16, 4, 128, 64, True, interleaved=True,
              fused=True),
        # a small fp32 run, as for checking gradients
        _rope("rope_fp32", "333", 4, 2, 64, 64, True, "f32", batch=2),
        # a decode step without the norm: q and k rotated, k and v into 16-bit pages
        _append("append_decode", ones, fill, 16, 4, 128, 128, 64, 16),
        # a serving batch's prompts of different lengths into fresh pages
        _append("append_prompt", "2048,1531,977,3200,64,411,1,2309", "0,0,0,0,0,0,0,0", 0, 4, 128,
                128, 64, 16, fused=True),
        # the next pieces of prompts into 4-bit pages, and all of their tokens back out
        _append("append_4bit", "512,300,2047", "8192,12001,77", 0, 4, 128, 128, 64, 4),
        # long prompts go on: their 16-bit pages as packed keys
        _gather("gather_prompt", "8192,12001,40001,5,700", 4, 128, 16, 16),
        # one user, one token
        _paged("paged_one", 1, 2048, 0.7, 1, 16, 2, 128, 64, 4),
        # a serving batch with rows of different lengths, in 4 and in 16 bits
        _paged("paged_batch_4bit", 64, 8192, 0.2, 1, 16, 4, 128, 64, 4),
        _paged("paged_batch", 64, 8192, 0.2, 1, 16, 4, 128, 16, 16),
        # one row with the million-token context
        _paged("paged_long_4bit", 1, 1 << 20, 0.95, 1, 16, 2, 128, 64, 4),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _cut(rng, total, n):
    cut = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cut, cut + [total])]


def _text(v):
    return ",".join(str(x) for x in v)


def draw(rng):
    op = rng.choice(["rope", "rope", "rope", "append", "append", "append", "gather", "paged",
                     "paged", "paged"])
    dtype = rng.choice(["bf16"] * 4 + ["f32"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 64, 96, 128, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    bits = 4 if rng.random() < 0.5 and D != 96 else {"bf16": 16, "f32": 32}[dtype]
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128])
        H = Hkv * rng.choice([1, 2, 4])
        R = rng.choice([D, D, D, D // 2 // 8 * 8, 0])
        norm = R == 0 or rng.random() < 0.7
        total = _log(rng, 1, max(2, (1 << (25 if dtype == "bf16" else 24)) // (D * (H + Hkv))))
        first = rng.choice([0, 0, _log(rng, 1, 100000)])
        more = dict(norm=norm, interleaved=rng.random() < 0.3, first=first, fused=rng.random() < 0.5)
        if rng.random() < 0.5:
            b = rng.choice([1, 2, 3, 16])
            return _rope(None, str(max(1, total // b)), H, Hkv, D, R, rng.random() < 0.6, dtype,
                         batch=b, **more)
        return _rope(None, _text(_cut(rng, total, min(total, rng.randint(1, 8)))), H, Hkv, D, R,
                     rng.random() < 0.6, dtype, **more)
    if op == "append":
        H = rng.choice([0, Hkv, 4 * Hkv])
        if rng.random() < 0.4:  # a decode step, or a few tokens of each row
            n = _log(rng, 1, 128)
            new = [rng.choice([1, 1, 3])] * n
        else:
            total = _log(rng, 20, 12000 if dtype == "bf16" else 6000)
            new = _cut(rng, total, min(total, rng.randint(1, 8)))
        used = [rng.choice([0, _log(rng, 1, 3000)]) for _ in new]
        return _append(None, _text(new), _text(used), H, Hkv, D, rng.choice([D, D, D // 2, 0]),
                       page, bits, dtype, rng.random() < 0.3, rng.random() < 0.5)
    if op == "gather":
        total = _log(rng, 50, 200000 // Hkv if dtype == "bf16" else 80000 // Hkv)
        return _gather(None, _text(_cut(rng, total, rng.randint(1, 8))), Hkv, D, page, bits, dtype)
    B = _log(rng, 1, 96)
    S = _log(rng, 70, min(300000, (1200000 if dtype == "bf16" else 300000) // (B * Hkv // 2 + 1)))
    return _paged(None, B, S, rng.choice([0.05, 0.5, 0.9]), rng.choice([1, 1, 1, 2, 4]),
                  Hkv * rng.choice([1, 2, 4, 8]), Hkv, D, page, bits, dtype)


def _ints(s):
    return [int(x) for x in str(s).split(",")]


def _fill(c):
    """The rows' tokens with the new ones: spread evenly over [used, 1] of S."""
    lo, hi = max(c["T"], int(c["used"] * c["S"])), max(c["T"], c["S"])
    return [hi - (hi - lo) * b // max(1, c["B"] - 1) for b in range(c["B"])] if c["B"] > 1 \
        else [(lo + hi) // 2]


def _token_bytes(c):
    """A cached token's k or v, all heads."""
    return c["Hkv"] * (c["D"] // 2 + c["D"] // GROUP * 2 if c["bits"] == 4
                       else c["D"] * c["bits"] // 8)


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        tokens = max(1, c["batch"]) * sum(_ints(c["lengths"]))
        n = tokens * (c["H"] + c["Hkv"]) * c["D"]
        rows = sum(_ints(c["lengths"]))  # of the tables
        return {"bytes": n * e * (5 if c["grad"] else 2) + rows * c["R"] * 4 + 8 * c["D"] * c["norm"],
                "flops": n * (24 if c["grad"] else 8)}
    if c["op"] == "append":
        n, new = c["Hkv"] * c["D"], sum(_ints(c["lengths"]))
        byts = new * (2 * n * e + 2 * _token_bytes(c) + 2 * c["H"] * c["D"] * e + c["R"] * 4)
        if c["bits"] == 4:  # and all tokens back out
            held = new + sum(_ints(c["used"]))
            byts += held * (2 * _token_bytes(c) + 4 * n)
        return {"bytes": byts, "flops": 12 * new * n}
    if c["op"] == "gather":
        n = sum(_ints(c["lengths"]))
        out = 2 if c["bits"] == 4 else e
        return {"bytes": n * (2 * _token_bytes(c) + 2 * c["Hkv"] * c["D"] * out),
                "flops": 2 * n * c["Hkv"] * c["D"]}
    keys = sum(_fill(c))
    return {"bytes": 2 * keys * _token_bytes(c) + 2 * c["B"] * c["T"] * c["H"] * c["D"] * e,
            "flops": 4 * c["D"] * c["H"] * c["T"] * keys}


# ------------------------------------------------------------------ inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(v):
    return _i32([sum(v[:i]) for i in range(len(v) + 1)])


def _tables(n, R):
    """cos and sin [n, R / 2] of position * 10000^(-2 i / R), made in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def _pages(c, held, g):
    """Pages with room for ``held[b]`` tokens per row, in no order, full of
    values; the table of each row's pages."""
    each = [-(-n // c["page"]) for n in held]
    most, total = max(each), sum(each) + 3
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.zeros(len(held), most, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    D, shape = c["D"], (total, c["Hkv"], c["page"])
    view = lambda x: x.transpose(1, 2)  # noqa: E731  a page's tokens of a head lie together
    if c["bits"] != 4:
        kv = [view(torch.randn(*shape, D, generator=g, device="cuda", dtype=TYPES[c["dtype"]]))
              for _ in range(2)]
        return kv, table
    cache = []
    for _ in range(2):  # codes of normal values whose steps are about 2.2 / 7 of their spread
        x = torch.randn(*shape, D, generator=g, device="cuda", dtype=torch.bfloat16)
        x = x.mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        codes = x[..., 0::2] | (x[..., 1::2] << 4)
        step = torch.randint(12, 29, (*shape, D // GROUP), generator=g, device="cuda")
        cache.append((view(codes), view((step / 64).to(torch.bfloat16))))
    return [cache[0][0], cache[1][0], cache[0][1], cache[1][1]], table


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)
    dt = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    st = {"c": c, "cos": None, "sin": None, "q": None}
    H, Hkv, D = c.get("H", 0), c["Hkv"], c["D"]
    if c["op"] == "rope":
        n = _ints(c["lengths"])
        B, T = max(1, c["batch"]), sum(n)
        if c["fused"]:
            qkv = normal(B, T, H + 2 * Hkv, D)
            st["q"], st["k"], _ = qkv.split([H, Hkv, Hkv], dim=2)
        else:
            st["q"], st["k"] = normal(B, T, H, D), normal(B, T, Hkv, D)
        st["wq"] = st["wk"] = st["positions"] = None
        if c["norm"]:
            st["wq"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
            st["wk"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        if c["R"]:
            st["cos"], st["sin"] = _tables(c["first"] + max(n), c["R"])
            if not c["batch"]:
                st["positions"] = torch.cat([torch.arange(c["first"], c["first"] + x, device="cuda")
                                             for x in n]).int()[None]
            elif c["first"]:  # rows that have come to different positions
                back = torch.randint(0, c["first"] + 1, (B, 1), generator=g, device="cuda")
                st["positions"] = (back + torch.arange(T, device="cuda")).int()
        if c["grad"]:
            st["dq"], st["dk"] = normal(B, T, H, D), normal(B, T, Hkv, D)
    elif c["op"] == "append":
        new, used = _ints(c["lengths"]), _ints(c["used"])
        held = [a + b for a, b in zip(new, used)]
        st["cache"], st["table"] = _pages(c, held, g)
        same = len(set(new)) == 1
        B, T = (len(new), new[0]) if same else (1, sum(new))
        if c["fused"]:
            qkv = normal(B, T, H + 2 * Hkv, D)
            st["q"], st["k"], st["v"] = qkv.split([H, Hkv, Hkv], dim=2)
        else:
            st["q"], st["k"], st["v"] = normal(B, T, H, D), normal(B, T, Hkv, D), normal(B, T, Hkv, D)
        if H == 0:
            st["q"] = None
        st["lens"] = _i32(used)
        st["cu"] = None if same else _offsets(new)
        if c["R"]:
            st["cos"], st["sin"] = _tables(max(held), c["R"])
        # for each new token its row and slot, as the plain form takes them
        row = torch.arange(len(new), device="cuda").repeat_interleave(torch.tensor(new, device="cuda"))
        st["row"], st["slot"] = row, torch.cat([torch.arange(a, a + b, device="cuda")
                                                for a, b in zip(used, new)])
        st["held"] = _offsets(held)
        st["total"] = sum(held)
    elif c["op"] == "gather":
        n = _ints(c["lengths"])
        st["cache"], st["table"] = _pages(c, n, g)
        st["held"], st["total"] = _offsets(n), sum(n)
    else:
        n = _fill(c)
        st["cache"], st["table"] = _pages(c, n, g)
        st["q"] = normal(c["B"], c["T"], H, D)
        st["lens"] = _i32([x - c["T"] for x in n])
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    import gated_delta_rule_bwd_gb300 as gdn

    c = st["c"]
    if c["op"] == "rope":
        how = dict(cos=st["cos"], sin=st["sin"], positions=st["positions"],
                   interleaved=c["interleaved"], eps=EPS)
        q, k = gdn.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], **how)
        out = {"q": q, "k": k}
        if c["grad"]:
            dq, dk, dwq, dwk = gdn.qk_norm_rope_bwd(st["q"], st["k"], st["dq"], st["dk"], st["wq"],
                                                    st["wk"], **how)
            out.update(dq=dq, dk=dk)
            if c["norm"]:
                out.update(dwq=dwq, dwk=dwk)
        return out
    if c["op"] == "append":
        q = gdn.kv_append(st["k"], st["v"], st["cache"], st["table"], st["lens"], q=st["q"],
                          cos=st["cos"], sin=st["sin"], interleaved=c["interleaved"],
                          cu_seqlens=st["cu"])
        out = {} if q is None else {"q": q}
        if c["bits"] == 4:
            out["k"], out["v"] = gdn.kv_gather(st["cache"], st["table"], st["held"], st["total"])
        else:
            out["k"], out["v"] = st["cache"]
        return out
    if c["op"] == "gather":
        k, v = gdn.kv_gather(st["cache"], st["table"], st["held"], st["total"])
        return {"k": k, "v": v}
    return {"o": gdn.attn_paged(st["q"], st["cache"], st["table"], st["lens"])}


# ------------------------------------------------------------------ the plain forms

def _rotate(x, cos, sin, interleaved, back=False):
    """x [..., heads, D] rotated by cos, sin [..., 1, R / 2]; fp32."""
    R = 2 * cos.shape[-1]
    s = -sin if back else sin
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * s, b * cos + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * s, b * cos + a * s], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_rope(x, w, cos, sin, interleaved, dy):
    n, r = x, None
    if w is not None:
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n = x * r * w
    y = n if cos is None else _rotate(n, cos, sin, interleaved)
    if dy is None:
        return y, None, None
    g = dy if cos is None else _rotate(dy, cos, sin, interleaved, back=True)
    if w is None:
        return y, g, None
    xh, u = x * r, g * w
    return y, r * (u - xh * (u * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1, 2))


def _quantise(x):
    """fp32 values [..., D] to codes and steps: a step per 32 values, the largest
    over 7 rounded to 5 significant bits."""
    x = x.unflatten(-1, (-1, GROUP))
    step = x.abs().amax(-1) * (1 / 7)
    step = step.view(torch.int32).add(0x40000).bitwise_and(-0x80000).view(torch.float32)
    s = step[..., None]
    n = torch.where(s > 0, x / s, torch.zeros_like(x)).round().clamp(-7, 7)
    n = n.add(8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), step.to(torch.bfloat16)


def _values(codes, step):
    """What 4-bit codes [..., D / 2] with steps [..., D / 32] stand for; fp32."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return (n.unflatten(-1, (-1, GROUP)) * step.float()[..., None]).flatten(-2)


def _taken(cache, at):
    """The cached k and v of the (page, place) pairs ``at``."""
    if len(cache) == 2:
        return cache[0][at], cache[1][at]
    return tuple(_values(cache[i][at], cache[2 + i][at]) for i in range(2))


def _held(st):
    """(page, place) of all tokens of all rows, one row after another."""
    cu, page = st["held"].long(), st["c"]["page"]
    i = torch.arange(st["total"], device="cuda")
    row = torch.bucketize(i, cu[1:], right=True)
    slot = i - cu[row]
    return st["table"].long()[row, slot // page], slot % page


def _run_plain(st):
    c = st["c"]
    dt = TYPES[c["dtype"]]
    if c["op"] == "rope":
        T = st["q"].shape[1]
        cos = sin = None
        if c["R"]:
            at = torch.arange(T, device="cuda")[None] if st["positions"] is None else st["positions"].long()
            cos, sin = st["cos"][at][:, :, None], st["sin"][at][:, :, None]
        grad = c["grad"]
        q, dq, dwq = _plain_rope(st["q"].float(), st["wq"], cos, sin, c["interleaved"],
                                 st["dq"].float() if grad else None)
        k, dk, dwk = _plain_rope(st["k"].float(), st["wk"], cos, sin, c["interleaved"],
                                 st["dk"].float() if grad else None)
        out = {"q": q.to(dt), "k": k.to(dt)}
        if grad:
            out.update(dq=dq.to(dt), dk=dk.to(dt))
            if c["norm"]:
                out.update(dwq=dwq, dwk=dwk)
        return out
    if c["op"] == "append":
        row, slot, cache = st["row"], st["slot"], st["cache"]
        at = st["table"].long()[row, slot // c["page"]], slot % c["page"]
        k, v = st["k"].flatten(0, 1).float(), st["v"].flatten(0, 1).float()
        q = None if st["q"] is None else st["q"].flatten(0, 1).float()
        if c["R"]:
            cos, sin = st["cos"][slot][:, None], st["sin"][slot][:, None]
            k = _rotate(k, cos, sin, c["interleaved"])
            q = None if q is None else _rotate(q, cos, sin, c["interleaved"])
        out = {} if q is None else {"q": q.to(dt).view(st["q"].shape)}
        if c["bits"] == 4:
            cache[0][at], cache[2][at] = _quantise(k)
            cache[1][at], cache[3][at] = _quantise(v)
            k, v = _taken(cache, _held(st))
            out.update(k=k.to(torch.bfloat16)[None], v=v.to(torch.bfloat16)[None])
        else:
            cache[0][at], cache[1][at] = k.to(dt), v.to(dt)
            out["k"], out["v"] = cache
        return out
    if c["op"] == "gather":
        k, v = _taken(st["cache"], _held(st))
        to = torch.bfloat16 if c["bits"] == 4 else dt
        return {"k": k.to(to)[None], "v": v.to(to)[None]}
    B, T, H, D = st["q"].shape
    Hkv = c["Hkv"]
    G = H // Hkv
    k, v = _taken(st["cache"], st["table"].long())  # [B, pages, page, Hkv, D]
    k, v = k.flatten(1, 2).float().permute(0, 2, 1, 3), v.flatten(1, 2).float().permute(0, 2, 1, 3)
    q = st["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    S = k.shape[2]
    last = st["lens"].long()[:, None] + torch.arange(T, device="cuda")[None, :]
    hide = torch.arange(S, device="cuda")[None, None, :] > last[:, :, None]
    hide = hide[:, None, None].expand(B, 1, G, T, S).reshape(B, 1, G * T, S)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).masked_fill_(hide, -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.div_(p.sum(-1, keepdim=True)), v)
    o = o.reshape(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, H, D)
    return {"o": o.to(dt)}


def run(st):
    return _run_own(st) if own else _run_plain(st)


# ------------------------------------------------------------------ 64 bits

def _turned(x, at, cos, sin, interleaved):
    """x [..., heads, D] in 64 bits: pairs as complex numbers times cos + i sin
    of the positions ``at``."""
    if cos is None:
        return x
    z = torch.complex(cos.double(), sin.double())[at][..., None, :]
    R = 2 * cos.shape[1]
    head, rest = x[..., :R], x[..., R:]
    if interleaved:
        y = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (R // 2, 2)).contiguous()) * z)
        return torch.cat([y.flatten(-2), rest], -1)
    y = torch.complex(head[..., :R // 2].contiguous(), head[..., R // 2:].contiguous()) * z
    return torch.cat([y.real, y.imag, rest], -1)


def _in_4_bits(x):
    """The values in 64 bits that 4-bit storage of x [..., D] stands for."""
    x = x.unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / 7)
    step = torch.ldexp(torch.floor(m * 32 + 0.5) / 32, e)
    n = torch.round(x / torch.where(step > 0, step, torch.ones_like(step))).clamp(-7, 7)
    return (n * step).flatten(-2)


def _row_pages(st, b, n):
    """The cached k and v of row b's first n tokens, in 64 bits."""
    pages = st["table"][b].long()[:-(-n // st["c"]["page"])]
    k, v = (x.flatten(0, 1)[:n].double() for x in
            (tuple(x[pages] for x in st["cache"][:2]) if len(st["cache"]) == 2 else
             tuple((lambda c, s: ((torch.stack([c % 16, c // 16], -1).flatten(-2).double() - 8)
                                  * s.double().repeat_interleave(GROUP, -1)))(x[pages], y[pages])
                   for x, y in zip(st["cache"][:2], st["cache"][2:]))))
    return k, v


def exact(c, seed):
    """The definitions in fp64; the gradients by differentiating the definition,
    not by its formulas."""
    st = prepare(c, seed)
    if c["op"] == "rope":
        res = {}
        T = st["q"].shape[1]
        at = torch.arange(T, device="cuda")[None] if st["positions"] is None else st["positions"].long()
        for n in ("q", "k"):
            x, w = st[n].double().requires_grad_(c["grad"]), st["w" + n]
            w = None if w is None else w.double().requires_grad_(c["grad"])
            y = x if w is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS) * w
            y = _turned(y, at, st["cos"], st["sin"], c["interleaved"])
            res[n] = y.detach()
            if c["grad"]:
                d = torch.autograd.grad(y, [x] if w is None else [x, w], st["d" + n].double())
                res["d" + n] = d[0]
                if w is not None:
                    res["dw" + n] = d[1]
        return res
    if c["op"] == "append":
        shape, res = st["k"].shape, {}
        at = st["slot"]
        turn = lambda x: _turned(x.double().flatten(0, 1), at, st["cos"], st["sin"], c["interleaved"])  # noqa: E731
        if st["q"] is not None:
            res["q"] = turn(st["q"]).view(st["q"].shape)
        new = {"k": turn(st["k"]), "v": st["v"].double().reshape(-1, *shape[2:])}
        counts, used = _ints(c["lengths"]), _ints(c["used"])
        if c["bits"] == 4:
            old = [_row_pages(st, b, n) if n else None for b, n in enumerate(used)]
            for i, n in enumerate(("k", "v")):
                parts = _in_4_bits(new[n]).split(counts)
                res[n] = torch.cat([x for b, p in enumerate(parts)
                                    for x in ([old[b][i], p] if old[b] else [p])])[None]
            return res
        for i, n in enumerate(("k", "v")):
            y = st["cache"][i].double()
            begin = 0
            for b, (m, u) in enumerate(zip(counts, used)):
                slots = torch.arange(u, u + m, device="cuda")
                y[st["table"][b].long()[slots // c["page"]], slots % c["page"]] = new[n][begin:begin + m]
                begin += m
            res[n] = y
        return res
    if c["op"] == "gather":
        rows = [_row_pages(st, b, n) for b, n in enumerate(_ints(c["lengths"]))]
        return {n: torch.cat([r[i] for r in rows])[None] for i, n in enumerate(("k", "v"))}
    B, T, H, D = st["q"].shape
    G = H // c["Hkv"]
    o = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        k, v = _row_pages(st, b, n + T)
        for t in range(T):
            q = st["q"][b, t].double().view(c["Hkv"], G, D)
            z = torch.einsum("hgd,nhd->hgn", q, k[:n + t + 1]) / math.sqrt(D)
            o[b, t] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), v[:n + t + 1]).reshape(H, D)
    return {"o": o}
