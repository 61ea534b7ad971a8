"""The training operators of the sparse-MoE layer, as they are timed and compared.

Grouped products by expert (forward and both gradients), SwiGLU with its
limit and routing weight (forward and backward) and the AdamW step over many
tensors. Each case runs either the plain form (elementary torch operations in
32 bits) or, with `own` set, the library's calls.

Sizes are those of the layer's own configurations: hidden 2560, expert width
768, 512 experts of which a token uses 8, batches of 1, 32 and 4096 tokens; a
share of 64 experts is what one of eight ranks holds under expert parallelism.
"""
import math
import random

import torch

own = False

H, I, E = 2560, 768, 512
BLOCK = 256            # elements that share a scale of the 8-bit states
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    def gl(name, op, rows, n, k, experts, skew, out="bf16", add=False, spare=0):
        return {"name": name, "op": op, "E": experts, "rows": rows, "N": n, "K": k, "skew": skew,
                "out": out, "add": add, "spare": spare}

    return [
        # one token's 8 gate rows: a decode step of a single sequence
        gl("linear_one_token", "linear", 8, I, H, E, 0.0),
        # the down product of a decode batch of 32 tokens
        gl("linear_decode", "linear", 256, H, I, E, 0.6),
        # the gate product of a 4096-token prefill, near-uniform loads: weight-bound
        gl("linear_prefill", "linear", 32768, I, H, E, 0.05),
        # the down product of one rank's 64 experts, uneven loads, a receive buffer with spare rows
        gl("linear_share", "linear", 30011, H, I, 64, 0.5, "bf16", False, 2757),
        # gradient of the gate product's input on one rank's share, and one summed onto another
        # branch's gradient with sizes that fill no tile
        gl("dgrad_share", "dgrad", 32768, I, H, 64, 0.3),
        gl("dgrad_ragged_add", "dgrad", 5003, 200, 1000, 32, 0.8, "fp32", True, 45),
        # gradient of the weights: one rank's share in 32 bits; all 512 experts, output-bound
        gl("wgrad_share", "wgrad", 32768, I, H, 64, 0.3, "fp32"),
        gl("wgrad_all_experts", "wgrad", 32768, I, H, E, 0.05),
        # between the products, 4096 tokens x 8 experts
        {"name": "swiglu_forward", "op": "swiglu", "rows": 32768, "I": I, "limit": 4.0,
         "weighted": True, "spare": 0},
        {"name": "swiglu_backward", "op": "swiglu_backward", "rows": 32001, "I": I, "limit": 7.0,
         "weighted": True, "spare": 767},
        # Wg, Wu and Wd of one rank's 64 experts with 8-bit states
        {"name": "adamw_experts_8bit", "op": "adamw", "sizes": "3x%d" % (64 * I * H), "p": "bf16",
         "master": False, "g": "bf16", "bits": 8},
        # router, bias and shared expert of 20 layers, master weights and states in 32 bits
        {"name": "adamw_dense_32bit", "op": "adamw",
         "sizes": "20x%d,20x%d,60x%d" % (E * H, E, I * H), "p": "bf16", "master": True,
         "g": "bf16", "bits": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "dgrad", "wgrad", "swiglu", "swiglu_backward", "adamw", "adamw"])
    if op in ("linear", "dgrad", "wgrad"):
        experts = rng.choice([8, 32, 64, 128, 256, 512])
        if rng.random() < 0.5:
            n, k = rng.choice([(I, H), (H, I)])
        else:  # any multiple of 8
            n = 8 * _log(rng, 8, 320)
            k = 8 * min(_log(rng, 8, 320), I * H // n // 8)
        skew = rng.choice([0.0, 0.1, 0.3, 0.6, 0.9])
        rows = _log(rng, 1, 32768)
        out = rng.choice(["bf16", "bf16", "fp32"])
        if op == "wgrad" and out == "fp32":
            experts = min(experts, 128)
        return {"op": op, "E": experts, "rows": rows, "N": n, "K": k, "skew": skew, "out": out,
                "add": out == "fp32" and rng.random() < 0.5,
                "spare": rng.choice([0, 0, _log(rng, 1, 2000)])}
    if op.startswith("swiglu"):
        return {"op": op, "rows": _log(rng, 1, 32768), "I": 8 * _log(rng, 8, 256),
                "limit": rng.choice([0.0, 4.0, 7.0]), "weighted": rng.random() < 0.7,
                "spare": rng.choice([0, _log(rng, 1, 2000)])}
    count, total = _log(rng, 1, 240), _log(rng, 20000, 100000000)
    small = 1 + _log(rng, 1, total // count)  # two kinds of tensors, as weights and biases
    large = total // count
    sizes = "%dx%d,%dx%d" % (count - count // 2, large, count // 2, small)
    p = rng.choice(["bf16", "fp32"])
    return {"op": "adamw", "sizes": sizes, "p": p, "master": p == "bf16" and rng.random() < 0.5,
            "g": rng.choice(["bf16", "fp32"]), "bits": rng.choice([8, 32])}


def _sizes(case):
    got = []
    for part in case["sizes"].split(","):
        c, n = part.split("x")
        got += [int(n)] * int(c)
    return got


def _counts(case, seed):
    """Rows of each expert: a popularity of uneven draws, every row independent."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    e, rows = case["E"], case["rows"]
    if rows <= 64 and case["skew"] == 0.0 and rows <= e:  # different experts, as top-k gives them
        counts = torch.zeros(e, dtype=torch.int64)
        counts[torch.randperm(e, generator=g)[:rows]] = 1
        return counts
    p = torch.exp(1.5 * case["skew"] * torch.randn(e, generator=g))
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=e)


def work(case):
    op = case["op"]
    if op in ("linear", "dgrad", "wgrad"):
        rows, n, k, experts = case["rows"], case["N"], case["K"], case["E"]
        touched = int((_counts(case, 1) > 0).sum())
        out = 2 if case["out"] == "bf16" else 4
        if case["add"]:
            out *= 2  # read and written
        if op == "linear":
            b = 2 * rows * k + 2 * touched * n * k + out * rows * n
        elif op == "dgrad":
            b = 2 * rows * n + 2 * touched * n * k + out * rows * k
        else:
            b = 2 * rows * (n + k) + out * (touched if case["add"] else experts) * n * k
        return {"bytes": b + 4 * (experts + 1), "flops": 2.0 * rows * n * k}
    if op == "swiglu":
        return {"bytes": 6.0 * case["rows"] * case["I"] + 8.0 * case["rows"] * case["weighted"],
                "flops": 8.0 * case["rows"] * case["I"]}
    if op == "swiglu_backward":
        return {"bytes": 10.0 * case["rows"] * case["I"] + 12.0 * case["rows"] * case["weighted"],
                "flops": 20.0 * case["rows"] * case["I"]}
    n = sum(_sizes(case))
    size = {"bf16": 2, "fp32": 4}
    per = size[case["g"]] + (2 + 8 if case["master"] else 2 * size[case["p"]])
    per += 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
    return {"bytes": per * n, "flops": 20.0 * n}


# ------------------------------------------------------------------ inputs
def _randn(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, bf = case["op"], torch.bfloat16
    st = {"case": case, "op": op}
    if op in ("linear", "dgrad", "wgrad"):
        counts = _counts(case, seed)
        n, k, experts = case["N"], case["K"], case["E"]
        cap = case["rows"] + case["spare"]
        offsets = torch.zeros(experts + 1, dtype=torch.int32)
        offsets[1:] = counts.cumsum(0)
        st["offsets"] = offsets.cuda()
        st["most"] = int(counts.max())
        st["touched"] = counts.nonzero()[:, 0].cuda()
        out = TYPES[case["out"]]
        if op != "dgrad":
            st["x"] = _randn((cap, k), gen, bf)
        if op != "linear":
            st["dy"] = _randn((cap, n), gen, bf, 0.02)
        if op != "wgrad":
            st["W"] = torch.empty(experts, n, k, dtype=bf, device="cuda")
            for e in range(0, experts, 64):
                m = min(64, experts - e)
                st["W"][e:e + m] = _randn((m, n, k), gen, bf, (k if op == "linear" else n) ** -0.5)
        shape = {"linear": (cap, n), "dgrad": (cap, k), "wgrad": (experts, n, k)}[op]
        st["out"] = _randn(shape, gen, out, 0.02) if case["add"] else torch.zeros(shape, dtype=out, device="cuda")
        if own:
            import sigmoid_group_limited_b200 as sgl
            st["ws"] = sgl.alloc_linear_workspace(experts, cap, n, k)
        return st
    if op.startswith("swiglu"):
        rows, cap, i = case["rows"], case["rows"] + case["spare"], case["I"]
        st["g"] = _randn((cap, i), gen, bf, 2.0)
        st["u"] = _randn((cap, i), gen, bf, 2.0)
        st["rows"] = torch.tensor([rows], dtype=torch.int32, device="cuda")
        st["w"] = st["perm"] = None
        if case["weighted"]:
            st["w"] = torch.rand(cap, device="cuda", generator=gen) * 0.6 + 0.05
            st["perm"] = torch.randperm(cap, device="cuda", generator=gen).to(torch.int32)
        zeros = lambda: torch.zeros(cap, i, dtype=bf, device="cuda")  # noqa: E731
        if op == "swiglu":
            st["h"] = zeros()
        else:
            st["dh"] = _randn((cap, i), gen, bf, 0.05)
            st["dg"], st["du"] = zeros(), zeros()
            st["dw"] = torch.zeros(cap, device="cuda") if case["weighted"] else None
        return st
    # AdamW: tensors lie in one buffer per kind, each from a multiple of BLOCK on
    sizes = _sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + BLOCK - 1) // BLOCK * BLOCK
    live = torch.ones(total, dtype=torch.bool, device="cuda")  # elements that belong to a tensor
    for s, n in zip(starts, sizes):
        if n % BLOCK:
            live[s + n:s + (n + BLOCK - 1) // BLOCK * BLOCK] = False
    p = _randn(total, gen, torch.float32, 0.03).mul_(live)
    st["p"] = p.to(TYPES[case["p"]])
    st["master"] = p.clone() if case["master"] else None
    scale = torch.exp(0.5 * torch.randn(total // BLOCK, 1, device="cuda", generator=gen)) * 1e-3
    noise = lambda: torch.randn(total // BLOCK, BLOCK, device="cuda", generator=gen)  # noqa: E731
    st["g"] = (noise() * scale).view(-1).mul_(live).to(TYPES[case["g"]])
    m = (noise() * 0.3 * scale).view(-1).mul_(live)
    v = ((noise() * 0.2).exp() * scale * scale).view(-1).mul_(live)
    del p, scale, live
    st["hyper"] = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 200}
    if case["bits"] == 32:
        st["m"], st["v"], st["ms"], st["vs"] = m, v, None, None
    else:
        st["m"], st["ms"] = _encode(m)
        st["v"], st["vs"] = _encode(v.sqrt_(), floor=True)
    if own:
        import sigmoid_group_limited_b200 as sgl

        def cut(t, s, n, per=1):
            return None if t is None else t[s // per:(s + n + per - 1) // per]

        st["tensors"] = sgl.make_adamw_tensors([
            dict(p=cut(st["p"], s, n), master=cut(st["master"], s, n), g=cut(st["g"], s, n),
                 m=cut(st["m"], s, n), v=cut(st["v"], s, n), m_scale=cut(st["ms"], s, n, BLOCK),
                 v_scale=cut(st["vs"], s, n, BLOCK)) for s, n in zip(starts, sizes)])
    return st


# ------------------------------------------------------------------ plain forms
def _padded(rows, lo, hi, most):
    """[segments, most, width] in 32 bits: each segment's rows, then zeros."""
    at = lo[:, None] + torch.arange(most, device=rows.device)[None, :]
    there = at < hi[:, None]
    got = rows[at.clamp_(max=rows.shape[0] - 1)].float()
    return got.mul_(there[:, :, None])


def _unpad_into(out, padded, lo, hi, add):
    """out[r] (+)= the padded row of r, for the rows that lie in a segment."""
    r = torch.arange(out.shape[0], device=out.device)
    e = torch.bucketize(r, hi, right=True)
    there = (e < padded.shape[0])[:, None]
    e = e.clamp_(max=padded.shape[0] - 1)
    at = (r - lo[e]).clamp_(max=padded.shape[1] - 1)
    new = padded[e, at]
    if add:
        new = new + out.float()
    out.copy_(torch.where(there, new, out.float()))


def _product_plain(st, rows, transpose):
    """rows of each touched expert times its matrix (or its transpose)."""
    t, off = st["touched"], st["offsets"].long()
    lo, hi = off[t], off[t + 1]
    w = (st["W"] if t.shape[0] == st["W"].shape[0] else st["W"][t]).float()
    y = torch.bmm(_padded(rows, lo, hi, st["most"]), w.transpose(1, 2) if transpose else w)
    _unpad_into(st["out"], y, lo, hi, st["case"]["add"])


def _wgrad_plain(st):
    off = st["offsets"].long()
    dy, x = (_padded(st[k], off[:-1], off[1:], st["most"]) for k in ("dy", "x"))
    y = torch.bmm(dy.transpose(1, 2), x)
    st["out"].copy_(y + st["out"].float() if st["case"]["add"] else y)


def _encode(v, floor=False):
    """Codes and scales of an 8-bit state: blocks of BLOCK elements over their
    largest magnitude, which becomes 448; with `floor`, what is not zero is at
    least the smallest code."""
    b = v.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    tiny = top < 2.0 ** -100
    scale = torch.where(tiny, 0.0, top / 448)
    y = b * torch.where(tiny, 0.0, 448 / top)
    q = y.to(F8)
    if floor:
        q = torch.where((y > 0) & (q.float() == 0), 2.0 ** -9, q.float()).to(F8)
    return q.view(-1), scale.view(-1)


def _decode(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw_plain(st):
    h = st["hyper"]
    g = st["g"].float()
    p = (st["master"] if st["master"] is not None else st["p"]).float()
    if st["ms"] is None:
        m, v = st["m"], st["v"]
    else:
        m, v = _decode(st["m"], st["ms"]), _decode(st["v"], st["vs"])
        v = v * v
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    root = v.sqrt()
    c1, c2 = 1 - h["beta1"] ** h["step"], math.sqrt(1 - h["beta2"] ** h["step"])
    p = p * (1 - h["lr"] * h["weight_decay"]) - (h["lr"] / c1) * (m / (root / c2 + h["eps"]))
    st["p"].copy_(p)
    if st["master"] is not None:
        st["master"].copy_(p)
    if st["ms"] is None:
        st["m"].copy_(m)
        st["v"].copy_(v)
    else:
        q, s = _encode(m)
        st["m"].copy_(q)
        st["ms"].copy_(s)
        q, s = _encode(root, floor=True)
        st["v"].copy_(q)
        st["vs"].copy_(s)


def _swiglu_parts(st):
    """Live rows: gate and up after the limit, their masks, sigmoid, the rows'
    slots and weights, in 32 bits."""
    n, lim = st["case"]["rows"], st["case"]["limit"]
    g, u = st["g"][:n].float(), st["u"][:n].float()
    lim = lim if lim > 0 else math.inf
    a, b = g.clamp(-lim, lim), u.clamp(-lim, lim)
    slot = st["perm"][:n].long() if st["perm"] is not None else None
    w = st["w"][slot][:, None] if slot is not None else 1.0
    return a, b, g.abs() <= lim, u.abs() <= lim, 1 / (1 + torch.exp(-a)), slot, w


def _swiglu_plain(st):
    a, b, _, _, s, _, w = _swiglu_parts(st)
    st["h"][:st["case"]["rows"]] = (w * a * s * b).to(torch.bfloat16)


def _swiglu_backward_plain(st):
    n = st["case"]["rows"]
    a, b, in_a, in_b, s, slot, w = _swiglu_parts(st)
    dh = st["dh"][:n].float()
    st["dg"][:n] = (w * dh * b * (s + a * s * (1 - s)) * in_a).to(torch.bfloat16)
    st["du"][:n] = (w * dh * (a * s) * in_b).to(torch.bfloat16)
    if slot is not None:
        st["dw"][slot] = (dh * (a * s * b)).sum(1)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        import sigmoid_group_limited_b200 as sgl
        if op == "linear":
            sgl.moe_grouped_linear(st["x"], st["offsets"], st["W"], st["out"], st["ws"], st["case"]["add"])
        elif op == "dgrad":
            sgl.moe_grouped_linear_dgrad(st["dy"], st["offsets"], st["W"], st["out"], st["ws"], st["case"]["add"])
        elif op == "wgrad":
            sgl.moe_grouped_linear_wgrad(st["dy"], st["x"], st["offsets"], st["out"], st["ws"], st["case"]["add"])
        elif op == "swiglu":
            sgl.moe_swiglu(st["g"], st["u"], st["h"], st["case"]["limit"], w=st["w"], perm=st["perm"], rows=st["rows"])
        elif op == "swiglu_backward":
            sgl.moe_swiglu_backward(st["dh"], st["g"], st["u"], st["dg"], st["du"], st["case"]["limit"], w=st["w"],
                                    perm=st["perm"], dw=st["dw"], rows=st["rows"])
        else:
            sgl.moe_adamw_step(st["tensors"], **st["hyper"])
    elif op == "linear":
        _product_plain(st, st["x"], True)
    elif op == "dgrad":
        _product_plain(st, st["dy"], False)
    elif op == "wgrad":
        _wgrad_plain(st)
    elif op == "swiglu":
        _swiglu_plain(st)
    elif op == "swiglu_backward":
        _swiglu_backward_plain(st)
    else:
        _adamw_plain(st)
    return _outputs(st)


def _outputs(st):
    op = st["op"]
    if op in ("linear", "dgrad", "wgrad"):
        return {"out": st["out"]}
    if op == "swiglu":
        return {"h": st["h"]}
    keys = ("dg", "du", "dw") if op == "swiglu_backward" else ("p", "master", "m", "v", "ms", "vs")
    return {k: st[k] for k in keys if st[k] is not None}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op in ("linear", "dgrad", "wgrad"):
        out = st["out"].to(d)
        base = out if case["add"] else torch.zeros((), dtype=d, device="cuda")
        off = st["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if op == "wgrad":
                got = st["dy"][lo:hi].to(d).t() @ st["x"][lo:hi].to(d)
                out[e] = got + (base[e] if case["add"] else 0)
            elif hi > lo:
                a, w = (st["x"], st["W"][e].t()) if op == "linear" else (st["dy"], st["W"][e])
                got = a[lo:hi].to(d) @ w.to(d)
                out[lo:hi] = got + (base[lo:hi] if case["add"] else 0)
        return {"out": out}
    if op.startswith("swiglu"):
        n, top = case["rows"], (case["limit"] or math.inf)
        g, u = (st[k][:n].to(d) for k in ("g", "u"))
        gate, up = torch.minimum(torch.maximum(g, g.new_tensor(-top)), g.new_tensor(top)), u.clamp(-top, top)
        sig = torch.sigmoid(gate)
        rows = torch.arange(n, device="cuda") if st["perm"] is None else st["perm"][:n].long()
        w = torch.ones(n, 1, dtype=d, device="cuda") if st["w"] is None else st["w"].to(d)[rows].unsqueeze(1)
        if op == "swiglu":
            h = st["h"].to(d)
            h[:n] = w * gate * sig * up
            return {"h": h}
        dh = st["dh"][:n].to(d)
        dg, du = st["dg"].to(d), st["du"].to(d)
        dg[:n] = torch.where(g.abs() <= top, w * dh * up * sig * (1 + gate * (1 - sig)), 0.0)
        du[:n] = torch.where(u.abs() <= top, w * dh * gate * sig, 0.0)
        if st["dw"] is None:
            return {"dg": dg, "du": du}
        dw = st["dw"].to(d)
        dw[rows] = (dh * gate * sig * up).sum(1)
        return {"dg": dg, "du": du, "dw": dw}
    # AdamW from the definition, the 8-bit states as codes of e4m3
    y = st["hyper"]
    p0 = (st["p"] if st["master"] is None else st["master"]).to(d)
    g = st["g"].to(d)
    if case["bits"] == 32:
        m, v = st["m"].to(d), st["v"].to(d)
    else:
        m = st["m"].to(d) * st["ms"].to(d).repeat_interleave(BLOCK)
        v = (st["v"].to(d) * st["vs"].to(d).repeat_interleave(BLOCK)) ** 2
    m = m * y["beta1"] + g * (1 - y["beta1"])
    v = v * y["beta2"] + g * g * (1 - y["beta2"])
    mh, vh = m / (1 - y["beta1"] ** y["step"]), v / (1 - y["beta2"] ** y["step"])
    p = p0 - y["lr"] * (mh / (vh.sqrt() + y["eps"]) + y["weight_decay"] * p0)
    out = {"p": p}
    if st["master"] is not None:
        out["master"] = p
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}
    for name, scale, t in (("m", "ms", m), ("v", "vs", v.sqrt())):
        b = t.view(-1, BLOCK)
        top = b.abs().max(1, keepdim=True).values
        s = torch.where(top < 2.0 ** -100, 0.0, top / 448)
        z = torch.where(s > 0, b / s, 0.0)
        mag = z.abs()
        # spacing of e4m3 at each magnitude: 2^(exponent - 3), 2^-9 below 2^-6
        step = torch.exp2(torch.frexp(mag.clamp(min=2.0 ** -6)).exponent.to(d) - 4)
        code = torch.round(mag / step) * step
        if name == "v":
            code = torch.where((mag > 0) & (code == 0), 2.0 ** -9, code)
        out[name], out[scale] = (code * z.sign()).view(-1), s.view(-1)
    return out
