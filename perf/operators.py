"""Workloads of the softmax-attention layer's operators and of layer norm.

A hybrid model puts causal attention layers between its linear-recurrent ones,
and a norm in front of every layer.  The cases here time those operators as a
program calls them:

  prompt   ``attn_fwd``: packed or batched prompts, also prompts that continue
           earlier keys;
  train    ``attn_fwd`` and ``attn_bwd``: one layer's attention in a step;
  decode   ``attn_decode``: one or a few new tokens per row against a cache;
  norm     ``layer_norm_fwd``, and with ``grad`` also ``layer_norm_bwd``.

With ``own`` false the same values come from elementary torch operations in
fp32, rounded once at the end.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _attn(name, op, lq, lk, H, Hkv, D, dtype="bf16", batch=0, fused=False):
    """``lq``/``lk``: lengths as text "5,37"; batch > 0: that many rows of one
    length; fused: q, k and v are views of one projection."""
    c = {"op": op, "lq": lq, "lk": lk, "H": H, "Hkv": Hkv, "D": D, "dtype": dtype, "batch": batch,
         "fused": fused}
    return dict(c, name=name) if name else c


def _decode(name, B, S, used, T, H, Hkv, D, dtype="bf16"):
    """B rows, caches of S slots, the rows' fill spread over [used, 1] of S."""
    c = {"op": "decode", "B": B, "S": S, "used": used, "T": T, "H": H, "Hkv": Hkv, "D": D,
         "dtype": dtype}
    return dict(c, name=name) if name else c


def _norm(name, rows, D, grad, dtype="bf16"):
    c = {"op": "norm", "rows": rows, "D": D, "grad": grad, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a short question among two shorter ones: latency
        _attn("prompt_short", "prompt", "5,61,33", "5,61,33", 8, 2, 128),
        # a serving batch's prompts of different lengths, packed; q, k, v from one projection
        _attn("prompt_packed", "prompt", "2048,1531,977,3200,64,411,1,2309",
              "2048,1531,977,3200,64,411,1,2309", 16, 4, 128, fused=True),
        # one long document
        _attn("prompt_long", "prompt", "16384", "16384", 16, 2, 128),
        # the next piece of two long prompts, against the keys that are there already
        _attn("prompt_continued", "prompt", "512,300", "8192,12001", 16, 4, 64),
        # attention layers in training, at the shape of the mixers' 300M workload
        _attn("train_300m", "train", "2048", "2048", 8, 8, 128, batch=16),
        # fine-tuning samples of different lengths packed into one row, grouped heads
        _attn("train_packed", "train", "3001,700,129,4096,15,251", "3001,700,129,4096,15,251",
              16, 4, 128, fused=True),
        # a small fp32 run, as for checking gradients
        _attn("train_fp32", "train", "333", "333", 4, 2, 64, "f32", batch=2),
        # one user, one token
        _decode("decode_one", 1, 2048, 0.7, 1, 16, 2, 128),
        # a serving batch with rows of different lengths
        _decode("decode_batch", 64, 8192, 0.2, 1, 16, 4, 128),
        # one row with the million-token context
        _decode("decode_long", 1, 1 << 20, 0.95, 1, 16, 2, 128),
        # the norm in front of a layer: a decode step's rows, and a training batch's
        _norm("norm_decode", 64, 2048, False),
        _norm("norm_train", 32768, 1024, True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _lengths(rng, total, n):
    cut = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cut, cut + [total])]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "train", "decode", "decode", "norm"])
    if op in ("prompt", "train"):
        f32 = rng.random() < 0.2
        Hkv = rng.choice([1, 2, 4] if f32 else [1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4] if Hkv < 8 else [1, 2])
        D = rng.choice([32, 64] if f32 else [64, 80, 96, 128, 128])
        total = _log(rng, 40, 1200 if f32 else 8400)
        if rng.random() < 0.35:
            b = rng.choice([1, 2, 3, 4])
            t = max(1, total // b)
            return _attn(None, op, str(t), str(t), H, Hkv, D, "f32" if f32 else "bf16", batch=b,
                         fused=rng.random() < 0.5)
        lq = _lengths(rng, total, rng.randint(1, 8))
        fused = rng.random() < 0.5
        lk = list(lq)
        if op == "prompt" and rng.random() < 0.4:  # a continued prompt: keys from before
            fused, lk = False, [x + _log(rng, 1, 2000) for x in lq]
        text = lambda v: ",".join(str(x) for x in v)  # noqa: E731
        return _attn(None, op, text(lq), text(lk), H, Hkv, D, "f32" if f32 else "bf16",
                     fused=fused)
    if op == "decode":
        f32 = rng.random() < 0.2
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 96)
        S = _log(rng, 70, min(300000, 1200000 // (B * Hkv // 2 + 1)))
        return _decode(None, B, S, rng.choice([0.05, 0.5, 0.9]), rng.choice([1, 1, 1, 2, 4]), H,
                       Hkv, rng.choice([64, 128, 128]), "f32" if f32 else "bf16")
    D = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 16, 1024), 1024, 2048])
    return _norm(None, _log(rng, 1, max(2, (1 << 25) // D)), D, rng.random() < 0.7,
                 rng.choice(["bf16", "bf16", "f32"]))


def _ints(s):
    return [int(x) for x in str(s).split(",")]


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("prompt", "train"):
        lq, lk = _ints(c["lq"]), _ints(c["lk"])
        n = max(1, c["batch"])
        pairs = n * c["H"] * sum(a * b - a * (a - 1) // 2 for a, b in zip(lq, lk))
        tq, tk = n * sum(lq), n * sum(lk)
        qb, kb = tq * c["H"] * c["D"] * e, tk * c["Hkv"] * c["D"] * e
        lse = tq * c["H"] * 4
        byts = 2 * qb + 2 * kb + lse  # q, k, v in; o, lse out
        flops = 4 * c["D"] * pairs
        if c["op"] == "train":  # and do in; dq, dk, dv out
            byts += 2 * qb + 2 * kb
            flops += 10 * c["D"] * pairs
        return {"bytes": byts, "flops": flops}
    if c["op"] == "decode":
        keys = sum(_fill(c))
        new = c["B"] * c["T"] * c["D"] * e
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * e + 2 * new * c["H"] + 4 * new * c["Hkv"],
                "flops": 4 * c["D"] * c["H"] * c["T"] * keys}
    n = c["rows"] * c["D"]
    return {"bytes": n * e * (5 if c["grad"] else 2) + 8 * c["D"] * (2 if c["grad"] else 1),
            "flops": n * (20 if c["grad"] else 8)}


def _fill(c):
    """The rows' tokens after the call: spread evenly over [used, 1] of the cache."""
    lo = max(1, int(c["used"] * c["S"]) - c["T"])
    hi = max(lo, c["S"] - c["T"])
    return [hi - (hi - lo) * b // max(1, c["B"] - 1) + c["T"] for b in range(c["B"])] \
        if c["B"] > 1 else [(lo + hi) // 2 + c["T"]]


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = TYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    st = {"c": c}
    if c["op"] in ("prompt", "train"):
        lq, lk = _ints(c["lq"]), _ints(c["lk"])
        B = max(1, c["batch"])
        tq, tk, H, Hkv, D = sum(lq), sum(lk), c["H"], c["Hkv"], c["D"]
        if c["fused"]:
            qkv = normal(B, tq, H + 2 * Hkv, D)
            st["q"], st["k"], st["v"] = qkv.split([H, Hkv, Hkv], dim=2)
        else:
            st["q"], st["k"], st["v"] = (normal(B, tq, H, D), normal(B, tk, Hkv, D),
                                         normal(B, tk, Hkv, D))
        if c["op"] == "train":
            st["do"] = normal(B, tq, H, D)
        st["lq"], st["lk"] = lq, lk
        cu = lambda v: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=torch.int32,  # noqa: E731
                                    device="cuda")
        st["cu"] = None if c["batch"] else cu(lq)
        st["cuk"] = None if c["batch"] or lk == lq else cu(lk)
    elif c["op"] == "decode":
        B, T, S, H, Hkv, D = c["B"], c["T"], c["S"], c["H"], c["Hkv"], c["D"]
        st["q"], st["k"], st["v"] = normal(B, T, H, D), normal(B, T, Hkv, D), normal(B, T, Hkv, D)
        st["k_cache"], st["v_cache"] = normal(B, S, Hkv, D), normal(B, S, Hkv, D)
        st["lens"] = torch.tensor([n - T for n in _fill(c)], dtype=torch.int32, device="cuda")
    else:
        st["x"] = normal(c["rows"], c["D"]) + 0.5
        st["w"] = 1 + 0.1 * torch.randn(c["D"], generator=g, device="cuda")
        st["b"] = 0.1 * torch.randn(c["D"], generator=g, device="cuda")
        if c["grad"]:
            st["dy"] = normal(c["rows"], c["D"])
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    import gated_delta_rule_bwd_gb300 as gdn

    c = st["c"]
    if c["op"] in ("prompt", "train"):
        o, lse = gdn.attn_fwd(st["q"], st["k"], st["v"], cu_seqlens=st["cu"],
                              cu_seqlens_k=st["cuk"])
        out = {"o": o, "lse": lse}
        if c["op"] == "train":
            dq, dk, dv = gdn.attn_bwd(st["q"], st["k"], st["v"], o, lse, st["do"],
                                      cu_seqlens=st["cu"], cu_seqlens_k=st["cuk"])
            out.update(dq=dq, dk=dk, dv=dv)
        return out
    if c["op"] == "decode":
        o = gdn.attn_decode(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["lens"])
        return {"o": o, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    y, mean, rstd = gdn.layer_norm_fwd(st["x"], st["w"], st["b"], eps=EPS)
    if not c["grad"]:
        return {"y": y}
    dx, dw, db = gdn.layer_norm_bwd(st["x"], st["w"], mean, rstd, st["dy"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


# ------------------------------------------------------------------ the plain forms

def _plain_attn(q, k, v, do=None, hide=None):
    """Rows of one length: q [B, lq, H, D], k, v [B, lk, Hkv, D], fp32; ``hide``
    [lq, lk] (default: the causal mask of one sequence).  The heads of a group
    are rows of one product with their shared key head."""
    B, lq, H, D = q.shape
    lk, Hkv = k.shape[1], k.shape[2]
    G, scale = H // Hkv, D ** -0.5
    rows = lambda x: x.reshape(B, lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * lq, D)  # noqa: E731
    back = lambda x: x.reshape(B, Hkv, G, lq, D).permute(0, 3, 1, 2, 4).reshape(B, lq, H, D)  # noqa: E731
    q2, k2, v2 = rows(q), k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    if hide is None:
        hide = (torch.arange(lk, device=q.device)[None, :]
                > torch.arange(lq, device=q.device)[:, None] + (lk - lq))
    hide = hide.repeat(G, 1)
    s = torch.matmul(q2, k2.transpose(-1, -2)).mul_(scale).masked_fill_(hide, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).reshape(B, Hkv, G, lq).reshape(B, H, lq)
    p = p.div_(total)
    o = torch.matmul(p, v2)
    if do is None:
        return back(o), lse
    do2 = rows(do)
    dv = torch.matmul(p.transpose(-1, -2), do2)
    ds = torch.matmul(do2, v2.transpose(-1, -2))
    ds = ds.sub_((do2 * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k2)
    dk = torch.matmul(ds.transpose(-1, -2), q2)
    return back(o), lse, back(dq), dk.permute(0, 2, 1, 3), dv.permute(0, 2, 1, 3)


def _packed_hide(tq, tk, cu, cuk):
    """The mask of all packed sequences in one [tq, tk] square."""
    i, j = torch.arange(tq, device=cu.device), torch.arange(tk, device=cu.device)
    si, sj = torch.bucketize(i, cu[1:], right=True), torch.bucketize(j, cuk[1:], right=True)
    last = i - cu[si] + (cuk[si + 1] - cuk[si]) - (cu[si + 1] - cu[si])
    return (si[:, None] != sj[None, :]) | ((j - cuk[sj])[None, :] > last[:, None])


def _run_plain(st):
    c = st["c"]
    dt = TYPES[c["dtype"]]
    if c["op"] in ("prompt", "train"):
        names = ("o", "lse", "dq", "dk", "dv") if c["op"] == "train" else ("o", "lse")
        x = [st[n].float() for n in ("q", "k", "v")]
        do = st["do"].float() if c["op"] == "train" else None
        tq, tk = x[0].shape[1], x[1].shape[1]
        if c["batch"]:
            parts = [_plain_attn(*x, do)]
        elif tq * tk <= 1 << 21:  # short sequences: one dense product costs less than many launches
            cuk = st["cu"] if st["cuk"] is None else st["cuk"]
            parts = [_plain_attn(*x, do, _packed_hide(tq, tk, st["cu"], cuk))]
        else:  # each sequence has scores of its own: one dense product over all would do more work
            cut = lambda t, n: t.split(n, dim=1)  # noqa: E731
            dos = cut(do, st["lq"]) if do is not None else [None] * len(st["lq"])
            parts = [_plain_attn(*a) for a in zip(cut(x[0], st["lq"]), cut(x[1], st["lk"]),
                                                  cut(x[2], st["lk"]), dos)]
        out = {n: torch.cat([p[i] for p in parts], dim=2 if n == "lse" else 1)
               for i, n in enumerate(names)}
        return {n: t.contiguous() if n == "lse" else t.to(dt).contiguous() for n, t in out.items()}
    if c["op"] == "decode":
        B, T, H, D = st["q"].shape
        S, Hkv = st["k_cache"].shape[1], st["k_cache"].shape[2]
        G = H // Hkv
        at = st["lens"].long()[:, None] + torch.arange(T, device="cuda")[None, :]
        row = torch.arange(B, device="cuda")[:, None]
        st["k_cache"][row, at] = st["k"]
        st["v_cache"][row, at] = st["v"]
        q = st["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
        k = st["k_cache"].float().permute(0, 2, 1, 3)
        v = st["v_cache"].float().permute(0, 2, 1, 3)
        hide = torch.arange(S, device="cuda")[None, None, :] > at[:, :, None]
        hide = hide[:, None, None].expand(B, 1, G, T, S).reshape(B, 1, G * T, S)
        s = torch.matmul(q, k.transpose(-1, -2)).mul_(D ** -0.5).masked_fill_(hide, -math.inf)
        p = s.sub_(s.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(p.div_(p.sum(-1, keepdim=True)), v)
        o = o.reshape(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, H, D)
        return {"o": o.to(dt), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    x = st["x"].float()
    d = x - x.mean(-1, keepdim=True)
    rstd = (d.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = d * rstd
    y = (xh * st["w"] + st["b"]).to(dt)
    if not c["grad"]:
        return {"y": y}
    dy = st["dy"].float()
    wdy = dy * st["w"]
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def run(st):
    return _run_own(st) if own else _run_plain(st)


# ------------------------------------------------------------------ 64 bits

def exact(c, seed):
    """The definitions in fp64, one key head of one sequence at a time; the
    gradients by differentiating the definition, not by its formulas."""
    st = prepare(c, seed)
    if c["op"] in ("prompt", "train"):
        B, tq, H, D = st["q"].shape
        Hkv = st["k"].shape[2]
        G = H // Hkv
        grad = c["op"] == "train"
        o = torch.zeros(B, tq, H, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H, tq, dtype=torch.float64, device="cuda")
        res = {"o": o, "lse": lse}
        if grad:
            res.update({"d" + n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda")
                        for n in ("q", "k", "v")})
        for b in range(B):
            for i in range(len(st["lq"])):
                q0, k0 = sum(st["lq"][:i]), sum(st["lk"][:i])
                lq, lk = st["lq"][i], st["lk"][i]
                see = torch.ones(lq, lk, dtype=torch.bool, device="cuda").tril(lk - lq)
                for h in range(H):
                    rows, keys = (b, slice(q0, q0 + lq)), (b, slice(k0, k0 + lk))
                    q = st["q"][rows][:, h].double().requires_grad_(grad)
                    k = st["k"][keys][:, h // G].double().requires_grad_(grad)
                    v = st["v"][keys][:, h // G].double().requires_grad_(grad)
                    s = torch.where(see, (q @ k.t()) / math.sqrt(D), -math.inf)
                    z = torch.logsumexp(s, 1)
                    y = torch.exp(s - z[:, None]) @ v
                    o[b, q0:q0 + lq, h], lse[b, h, q0:q0 + lq] = y.detach(), z.detach()
                    if grad:
                        d = torch.autograd.grad(y, (q, k, v), st["do"][rows][:, h].double())
                        res["dq"][b, q0:q0 + lq, h] = d[0]
                        res["dk"][b, k0:k0 + lk, h // G] += d[1]
                        res["dv"][b, k0:k0 + lk, h // G] += d[2]
        return res
    if c["op"] == "decode":
        B, T, H, D = st["q"].shape
        G = H // st["k"].shape[2]
        o = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens"].tolist()):
            for h in range(H // G):
                k = torch.cat([st["k_cache"][b, :n, h], st["k"][b, :, h]]).double()
                v = torch.cat([st["v_cache"][b, :n, h], st["v"][b, :, h]]).double()
                for t in range(T):
                    z = st["q"][b, t, h * G:(h + 1) * G].double() @ k[:n + t + 1].t()
                    o[b, t, h * G:(h + 1) * G] = torch.softmax(z / math.sqrt(D), -1) @ v[:n + t + 1]
        return {"o": o, "k_cache": None, "v_cache": None}
    grad = c["grad"]
    x = st["x"].double().requires_grad_(grad)
    w, b = st["w"].double().requires_grad_(grad), st["b"].double().requires_grad_(grad)
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    y = (x - mean) / torch.sqrt(var + EPS) * w + b
    if not grad:
        return {"y": y}
    dx, dw, db = torch.autograd.grad(y, (x, w, b), st["dy"].double())
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}
