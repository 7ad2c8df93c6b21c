"""What stands around an expert layer, as timed cases: residual add + layer norm
and its gradient, the experts' FFN in 8-bit integers, and the global gradient
norm with clipping.

Each case has two forms on the same inputs. With `own` false, `run` computes it
in elementary torch operations (32-bit, rounded once at the end; 64-bit for long
sums); with `own` true, it makes the library's calls. `exact` states the same
operator in 64 bits, written apart from both.

Formulas
  norm       s = x + r (rounded to x's type; s = x without r), m = mean(s),
             v = mean((s - m)^2), rstd = 1 / sqrt(v + eps),
             y = (s - m) * rstd * w + b
  norm_bwd   h = (s - m) * rstd, g = w * dy,
             dx = rstd * (g - mean(g) - h * mean(g * h)) + ds,
             dw = sum over rows of dy * h, db = sum over rows of dy
  int8       per local row a = x[perm / k]: scale = max(max|a| / 127, 2^-126),
             q = rint(a / scale); [G | U] = (q . Wq) * scale * channel scale;
             h = silu(G) * U in x's type, quantised in the same way; y = (hq . Wq2)
             * scale * channel scale
  grad_norm  norm = sqrt(sum over all tensors of g^2)
  clip       out = g * min(1, max_norm / (norm + 1e-6))
"""
import math
import random

import torch

own = False

_EPS = 1e-5
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode batch's hidden states: launch latency
        dict(name="norm_decode", op="norm", T=32, d=2880, dtype="bf16", wdtype="bf16", bias=True, residual=True),
        # the longest prompt batch with the widest rows
        dict(name="norm_wide", op="norm", T=16384, d=7168, dtype="bf16", wdtype="bf16", bias=True, residual=True),
        # fp32 throughout, a ragged batch of narrow rows, no bias, no residual
        dict(name="norm_narrow_f32", op="norm", T=5003, d=136, dtype="f32", wdtype="f32", bias=False, residual=False),
        # a training step's norm gradient with the residual stream's gradient added, fp32 norm weights
        dict(name="norm_bwd_train", op="norm_bwd", T=4096, d=4096, dtype="bf16", wdtype="f32", bias=True,
             residual=True),
        # the same without the residual stream, a ragged batch
        dict(name="norm_bwd_ragged", op="norm_bwd", T=777, d=2880, dtype="bf16", wdtype="bf16", bias=True,
             residual=False),
        # single-token serving: 32 sequences over 128 local experts, expert weights streamed once
        dict(name="int8_decode32", op="int8", T=32, d=2880, d_ff=2880, E=128, k=4, e_begin=0, e_end=128,
             dtype="bf16"),
        # one sequence's token, small experts with ragged widths: launch latency
        dict(name="int8_one_token", op="int8", T=1, d=1000, d_ff=1480, E=32, k=4, e_begin=0, e_end=32,
             dtype="bf16"),
        # one rank's share of a 128-expert layer, a prompt batch
        dict(name="int8_share128", op="int8", T=8192, d=2880, d_ff=2880, E=128, k=4, e_begin=0, e_end=16,
             dtype="bf16"),
        # 8 experts, all local: the largest products
        dict(name="int8_dense8", op="int8", T=4096, d=4096, d_ff=14336, E=8, k=2, e_begin=0, e_end=8,
             dtype="bf16"),
        # the norm alone, before a sum over ranks: a rank's share of fp32 expert gradients
        dict(name="grad_norm_share128", op="grad_norm", count=2, largest=16 * 2880 * 5760, smallest=16 * 2880 * 2880,
             dtype="f32", flat=False, std=1e-3, max_norm=1.0),
        # the whole clip over 8 experts' bf16 weight gradients
        dict(name="clip_dense8", op="clip", count=2, largest=8 * 4096 * 28672, smallest=8 * 14336 * 4096,
             dtype="bf16", flat=False, std=1e-3, max_norm=1.0),
        # many small parameters (norm weights, biases, routers), views of one flat buffer at odd offsets
        dict(name="clip_many_small", op="clip", count=60, largest=368641, smallest=1, dtype="f32", flat=True,
             std=1e-2, max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "int8", "int8", "grad_norm", "clip"])
    while True:
        if op in ("norm", "norm_bwd"):
            dtype = rng.choice(["bf16", "bf16", "f32"])
            case = dict(op=op, T=_log_int(rng, 1, 16384), d=8 * _log_int(rng, 1, 2048), dtype=dtype,
                        wdtype=rng.choice([dtype, "f32"]), bias=rng.random() < 0.7, residual=rng.random() < 0.6)
            ok = case["T"] * case["d"] * _BYTES[dtype] <= 16384 * 7168 * 2
        elif op == "int8":
            E = rng.choice([4, 8, 16, 32, 64, 128, 256])
            e_loc = rng.choice([v for v in (E, E // 2, E // 4, E // 8) if v >= 1])
            e_begin = e_loc * rng.randrange(E // e_loc)
            case = dict(op=op, T=_log_int(rng, 1, 8192), d=8 * _log_int(rng, 8, 512), d_ff=8 * _log_int(rng, 8, 1792),
                        E=E, k=rng.randint(1, min(8, E)), e_begin=e_begin, e_end=e_begin + e_loc,
                        dtype="bf16")
            w = work(case)
            ok = w["flops"] <= 6 * 8192 * 4096 * 14336 and 3 * e_loc * case["d"] * case["d_ff"] <= 3 * 8 * 4096 * 14336
        else:
            smallest = _log_int(rng, 1, 1 << 20)
            case = dict(op=op, count=_log_int(rng, 1, 200), largest=_log_int(rng, smallest, 1 << 27), smallest=smallest,
                        dtype=rng.choice(["bf16", "f32", "mixed"]), flat=rng.random() < 0.5,
                        std=rng.choice([1e-6, 1e-3, 1e-1]), max_norm=rng.choice([0.5, 1.0, 10.0]))
            ok = sum(_sizes(case)) <= 3 * 8 * 4096 * 14336 // 2
        if ok:
            return case


# --------------------------------------------------------------------- the work

def _counts(case):
    """Expected local pairs and local experts with at least one row, for uniform routing."""
    T, E, k, e_loc = case["T"], case["E"], case["k"], case["e_end"] - case["e_begin"]
    return T * k * e_loc / E, e_loc * (1.0 - (1.0 - k / E) ** T)


def _sizes(case):
    """Element counts of the tensors: the largest, the smallest, the rest log-uniform between."""
    rng = random.Random(f"{case['count']}/{case['largest']}/{case['smallest']}")
    mid = [_log_int(rng, case["smallest"], case["largest"]) for _ in range(max(0, case["count"] - 2))]
    return [case["largest"]] + mid + ([case["smallest"]] if case["count"] > 1 else [])


def _types(case):
    n = case["count"]
    return [("bf16", "f32")[i % 2] if case["dtype"] == "mixed" else case["dtype"] for i in range(n)]


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, d, b, wb = case["T"], case["d"], _BYTES[case["dtype"]], _BYTES[case["wdtype"]]
        params = d * wb * (2 if case["bias"] else 1)
        if op == "norm":  # x (and r) read, y (and s) written, two fp32 statistics a row
            return dict(bytes=T * d * b * (4 if case["residual"] else 2) + 8 * T + params,
                        flops=T * d * (9 if case["residual"] else 8))
        return dict(bytes=T * d * b * (4 if case["residual"] else 3) + 8 * T + d * wb + params, flops=T * d * 15)
    if op == "int8":
        n_loc, active = _counts(case)
        d, f, b = case["d"], case["d_ff"], _BYTES[case["dtype"]]
        return dict(bytes=active * (3.0 * d * f + 4 * (2 * f + d)) + min(case["T"], n_loc) * d * b + n_loc * d * b
                    + 4 * case["T"] * case["k"],
                    flops=6.0 * n_loc * d * f)
    sizes, total = _sizes(case), 0
    for n, t in zip(sizes, _types(case)):
        total += n * _BYTES[t]
    if op == "grad_norm":
        return dict(bytes=total + 4, flops=2 * sum(sizes))
    return dict(bytes=2 * total + 4, flops=3 * sum(sizes))


# -------------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1 + 7919 * seed)
    op = case["op"]

    def normal(shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).add_(mean).to(dtype)

    if op in ("norm", "norm_bwd"):
        T, d, dt, wdt = case["T"], case["d"], _DT[case["dtype"]], _DT[case["wdtype"]]
        # a residual stream's rows: a few large channels, and a mean off zero
        chan = torch.exp(normal((d,), 0.5))
        x = (normal((T, d)) * chan + 0.25).to(dt)
        st = dict(case=case, x=x, w=normal((d,), 0.2, 1.0, wdt), b=normal((d,), 0.1, 0.0, wdt) if case["bias"] else None)
        if op == "norm":
            st["r"] = normal((T, d), 0.5, 0.0, dt) if case["residual"] else None
        else:
            f = x.double()
            mean = f.mean(dim=1)
            st["mean"] = mean.float()
            st["rstd"] = (1.0 / torch.sqrt(((f - mean[:, None]) ** 2).mean(dim=1) + _EPS)).float()
            st["dy"] = normal((T, d), 1.0, 0.0, dt)
            st["ds"] = normal((T, d), 1.0, 0.0, dt) if case["residual"] else None
        return st
    if op == "int8":
        return _prepare_int8(case, normal, dev)
    sizes, types = _sizes(case), _types(case)
    grads, outs = [], []
    for t in ("bf16", "f32"):
        mine = [i for i in range(len(sizes)) if types[i] == t]
        if case["flat"]:  # one flat buffer of each type, the tensors are consecutive views of it
            total = sum(sizes[i] for i in mine)
            fg, fo = torch.empty(total, dtype=_DT[t], device=dev), torch.empty(total, dtype=_DT[t], device=dev)
            at = 0
            for i in mine:
                grads.append((i, fg[at:at + sizes[i]]))
                outs.append((i, fo[at:at + sizes[i]]))
                at += sizes[i]
        else:
            for i in mine:
                grads.append((i, torch.empty(sizes[i], dtype=_DT[t], device=dev)))
                outs.append((i, torch.empty(sizes[i], dtype=_DT[t], device=dev)))
    grads = [g for _, g in sorted(grads, key=lambda p: p[0])]
    outs = [g for _, g in sorted(outs, key=lambda p: p[0])]
    for i, g in enumerate(grads):  # each parameter has its own gradient scale
        std = case["std"] * 2.0 ** ((i * 5) % 7 - 3)
        for at in range(0, g.numel(), 1 << 28):
            part = g[at:at + (1 << 28)]
            part.copy_(torch.randn(part.numel(), generator=gen, device=dev).mul_(std))
    return dict(case=case, grads=grads, outs=outs)


def _prepare_int8(case, normal, dev):
    T, d, f, E, k = case["T"], case["d"], case["d_ff"], case["E"], case["k"]
    lo, hi, dt = case["e_begin"], case["e_end"], _DT[case["dtype"]]
    e_loc = hi - lo
    x = normal((T, d), 1.0, 0.0, dt)
    idx = torch.topk(normal((T, E)), k, dim=1).indices.reshape(-1)
    perm = torch.sort(idx, stable=True).indices.to(torch.int32)
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)

    def weight(K, N):
        """[e_loc, ceil(K / 64), N, 64] int8 (64 consecutive K values of a channel together, zeros past K)
        and the channels' scales [e_loc, N]."""
        kb = (K + 63) // 64
        q = torch.empty((e_loc, kb, N, 64), dtype=torch.int8, device=dev)
        for e in range(e_loc):
            q[e] = torch.round(normal((kb, N, 64), 30.0)).clamp_(-127, 127).to(torch.int8)
            if K % 64:
                q[e, -1, :, K % 64:] = 0
        scale = (0.8 + 0.4 * torch.sigmoid(normal((e_loc, N)))) / (30.0 * math.sqrt(K))
        return q, scale

    wgu, sgu = weight(d, 2 * f)
    wdn, sdn = weight(f, d)
    y = torch.zeros((T * min(k, e_loc), d), dtype=dt, device=dev)
    return dict(case=case, x=x, perm=perm, offsets=offsets, wgu=wgu, sgu=sgu, wdn=wdn, sdn=sdn, y=y,
                bounds=[int(v) for v in offsets.cpu()])


# ------------------------------------------------------------------------ a pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own[op](state)
    return _plain[op](state)


def _plain_norm(st):
    x = st["x"]
    s = x if st["r"] is None else (x.float() + st["r"].float()).to(x.dtype)
    f = s.float()
    mean = f.mean(dim=1)
    c = f - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1) + _EPS)
    y = c * rstd[:, None] * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    return [y.to(x.dtype), s, mean, rstd]


def _plain_norm_bwd(st):
    x = st["x"]
    dy = st["dy"].float()
    h = (x.float() - st["mean"][:, None]) * st["rstd"][:, None]
    g = dy * st["w"].float()
    dx = st["rstd"][:, None] * (g - g.mean(dim=1, keepdim=True) - h * (g * h).mean(dim=1, keepdim=True))
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
    out = [dx.to(x.dtype), (dy * h).sum(dim=0).to(st["w"].dtype)]
    if st["b"] is not None:
        out.append(dy.sum(dim=0).to(st["w"].dtype))
    return out


def _quantize_rows(a):
    a = a.float()
    scale = torch.clamp(a.abs().amax(dim=1) / 127.0, min=2.0 ** -126)
    return torch.round(a * (1.0 / scale)[:, None]), scale


def _plain_int8(st):
    c, y = st["case"], st["y"]
    d, f, k = c["d"], c["d_ff"], c["k"]
    b0 = st["bounds"][c["e_begin"]]
    q, scale = _quantize_rows(st["x"])
    for e in range(c["e_end"] - c["e_begin"]):
        r0, r1 = st["bounds"][c["e_begin"] + e], st["bounds"][c["e_begin"] + e + 1]
        if r0 == r1:
            continue
        tok = (st["perm"][r0:r1] // k).long()
        w = st["wgu"][e].permute(0, 2, 1).reshape(-1, 2 * f)[:d].float()
        gu = (q[tok] @ w) * st["sgu"][e] * scale[tok][:, None]
        h = (gu[:, :f] / (1.0 + torch.exp(-gu[:, :f])) * gu[:, f:]).to(y.dtype)
        hq, hs = _quantize_rows(h)
        w = st["wdn"][e].permute(0, 2, 1).reshape(-1, d)[:f].float()
        y[r0 - b0:r1 - b0] = ((hq @ w) * st["sdn"][e] * hs[:, None]).to(y.dtype)
    return y


def _plain_grad_norm(st):
    total = torch.zeros((), dtype=torch.float64, device=st["grads"][0].device)
    for g in st["grads"]:
        f = g.double()
        total = total + (f * f).sum()
    return torch.sqrt(total).float().reshape(1)


def _plain_clip(st):
    norm = _plain_grad_norm(st)
    coef = torch.clamp(st["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    for g, o in zip(st["grads"], st["outs"]):
        o.copy_((g.float() * coef).to(g.dtype))
    return [norm] + st["outs"]


_plain = dict(norm=_plain_norm, norm_bwd=_plain_norm_bwd, int8=_plain_int8, grad_norm=_plain_grad_norm,
              clip=_plain_clip)


def _own_norm(st):
    import token_dispatch_grouped_amd as moe
    y, s, mean, rstd = moe.layer_norm(st["x"], st["w"], st["b"], eps=_EPS, residual=st["r"])
    return [y, s, mean, rstd]


def _own_norm_bwd(st):
    import token_dispatch_grouped_amd as moe
    dx, dw, db = moe.layer_norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], d_s=st["ds"],
                                         bias=st["b"] is not None)
    return [dx, dw] if db is None else [dx, dw, db]


def _own_int8(st):
    import token_dispatch_grouped_amd as moe
    c = st["case"]
    experts = moe.Int8Experts(st["wgu"], st["sgu"], st["wdn"], st["sdn"])
    return moe.grouped_gemm_int8(st["x"], st["perm"], st["offsets"], experts, c["k"], c["E"], c["e_begin"], c["e_end"],
                                 y=st["y"])


def _own_grad_norm(st):
    import token_dispatch_grouped_amd as moe
    return moe.grad_norm(st["grads"])


def _own_clip(st):
    import token_dispatch_grouped_amd as moe
    norm = moe.clip_grad_norm(st["grads"], st["case"]["max_norm"], out=st["outs"])
    return [norm] + st["outs"]


_own = dict(norm=_own_norm, norm_bwd=_own_norm_bwd, int8=_own_int8, grad_norm=_own_grad_norm, clip=_own_clip)


# ------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s = st["x"].double()
        if st["r"] is not None:  # the sum is held in x's type: the rest of the operator starts from it
            s = (s + st["r"].double()).to(st["x"].dtype).double()
        var, mean = torch.var_mean(s, dim=1, correction=0)
        rstd = torch.rsqrt(var + _EPS)
        y = torch.addcmul(torch.zeros_like(s) if st["b"] is None else st["b"].double().expand_as(s),
                          (s - mean.unsqueeze(1)) * rstd.unsqueeze(1), st["w"].double().expand_as(s))
        return [y, s, mean, rstd]
    if op == "norm_bwd":
        dy, w = st["dy"].double(), st["w"].double()
        mean, rstd = st["mean"].double().unsqueeze(1), st["rstd"].double().unsqueeze(1)
        h = (st["x"].double() - mean) * rstd
        n = case["d"]
        first = torch.mv(dy, w).unsqueeze(1) / n
        second = torch.mv(dy * h, w).unsqueeze(1) / n
        dx = (dy * w - first - h * second) * rstd
        if st["ds"] is not None:
            dx += st["ds"].double()
        out = [dx, torch.multiply(dy, h, out=h).sum(dim=0)]
        return out + [dy.sum(dim=0)] if case["bias"] else out
    if op == "int8":
        return _exact_int8(case, st)
    total = 0.0
    for g in st["grads"]:
        for at in range(0, g.numel(), 1 << 27):
            part = g[at:at + (1 << 27)].double()
            total += float(torch.dot(part, part))
    norm = math.sqrt(total)
    if op == "grad_norm":
        return torch.tensor([norm], dtype=torch.float64)
    coef = min(1.0, case["max_norm"] / (norm + 1e-6))
    return [torch.tensor([norm], dtype=torch.float64)] + [g.double() * coef for g in st["grads"]]


def _exact_int8(case, st):
    d, f, lo, hi = case["d"], case["d_ff"], case["e_begin"], case["e_end"]
    offs = st["offsets"].cpu().tolist()
    rows = torch.div(st["perm"][offs[lo]:offs[hi]].long(), case["k"], rounding_mode="floor")
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=st["y"].device)

    def codes(a):
        step = torch.clamp_min(a.abs().max(dim=1, keepdim=True).values / 127, 2.0 ** -126)
        return torch.round(a / step), step

    def matrix(q, scale, e, K):
        m = q[e].transpose(0, 1).reshape(q.shape[2], -1)[:, :K].double() * scale[e].double().unsqueeze(1)
        return m.t().contiguous()

    for e in range(lo, hi):
        mine = rows[offs[e] - offs[lo]:offs[e + 1] - offs[lo]]
        if mine.numel() == 0:
            continue
        q, step = codes(st["x"].index_select(0, mine).double())
        both = (q * step) @ matrix(st["wgu"], st["sgu"], e - lo, d)
        gate, up = both.split(f, dim=1)
        h = (gate * torch.sigmoid(gate) * up).to(st["x"].dtype).double()  # held in x's type between the products
        hq, hstep = codes(h)
        y[offs[e] - offs[lo]:offs[e + 1] - offs[lo]] = (hq * hstep) @ matrix(st["wdn"], st["sdn"], e - lo, f)
    return y
