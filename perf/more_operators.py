"""What a step of an expert layer needs next to the layer itself, as timed cases:
routing by scores, RMS norm with the residual's addition (and 8-bit rows for the
experts) and its gradient, and the AdamW step over many tensors with states in 32
or 8 bits.

Each case has two forms on the same inputs. With `own` false, `run` computes it
in elementary torch operations (32-bit, rounded once at the end; 64-bit where an
order hangs on it); with `own` true, it makes the library's calls. `exact` states
the same operator in 64 bits, written apart from both.

Formulas
  route      s = softmax(x) or sigmoid(x); the choice goes by c = s + bias, rounded
             to 32 bits (by x itself without a bias and without groups); of the
             groups of experts the top_groups with the largest sum of their two
             largest c stay; idx = the k largest c of those, ties to the lower id;
             w = scale * s[idx], or scale * s[idx] / sum(s[idx])
  route_bwd  the gradient of w with respect to x for given idx (no gradient passes
             through the choice)
  rms        s = x + r (rounded to x's type; s = x without r),
             rstd = 1 / sqrt(mean(s^2) + eps), y = s * rstd * w; 8-bit rows:
             scale = max(max|y| / 127, 2^-126), q = rint(y * (1 / scale))
  rms_bwd    h = s * rstd, g = w * dy, dx = rstd * (g - h * mean(g * h)) + ds,
             dw = sum over rows of dy * h
  adamw      g = grad * min(1, max_norm / (norm + 1e-6)); m = b1 m + (1 - b1) g;
             v = b2 v + (1 - b2) g^2; p = p - lr wd p
             - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
  adamw8     the same with m and sqrt(v) held as e4m3 codes, a scale for each 128
             elements: scale = max(max / 448, 2^-126), code = e4m3(value * (1 / scale)),
             and at least 2^-9 for a root above zero
"""
import math
import random

import torch

own = False

_EPS = 1e-6
_LR, _B1, _B2, _AEPS, _WD, _STEP = 3e-5, 0.9, 0.95, 1e-8, 0.1, 1000
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_BLOCK = 128  # elements with one scale in an 8-bit state


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode batch's tokens over 128 experts: launch latency
        dict(name="route_decode", op="route", T=32, E=128, k=4, score="softmax", bias=False, groups=1, top_groups=1,
             renormalize=True, scale=1.0, held="f32"),
        # a prompt batch over 256 experts in 8 groups, sigmoid scores with a balance bias, logits from a bf16 product
        dict(name="route_prompt", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renormalize=True, scale=2.5, held="bf16"),
        # the same batch's gradient in training
        dict(name="route_bwd_train", op="route_bwd", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renormalize=True, scale=2.5, held="f32"),
        # softmax weights that are not renormalised (every logit has a gradient), a ragged batch and expert count
        dict(name="route_bwd_ragged", op="route_bwd", T=5003, E=60, k=4, score="softmax", bias=False, groups=1,
             top_groups=1, renormalize=False, scale=1.0, held="f32"),
        # one decode batch's hidden states, normalised into bf16 for the router and 8-bit rows for the experts
        dict(name="rms_decode_int8", op="rms", T=32, d=2880, dtype="bf16", wdtype="bf16", residual=True, int8=True),
        # the longest prompt batch with the widest rows
        dict(name="rms_prompt", op="rms", T=16384, d=7168, dtype="bf16", wdtype="bf16", residual=True, int8=False),
        # a training step's norm gradient with the residual stream's gradient added, fp32 norm weights
        dict(name="rms_bwd_train", op="rms_bwd", T=4096, d=4096, dtype="bf16", wdtype="f32", residual=True),
        # fp32 throughout, a ragged batch, no residual stream
        dict(name="rms_bwd_ragged_f32", op="rms_bwd", T=777, d=2888, dtype="f32", wdtype="f32", residual=False),
        # a rank's 16 experts (gate/up and down weights): bf16 weights with fp32 masters, 32-bit states
        dict(name="adamw_share128", op="adamw", count=2, largest=16 * 2880 * 5760, smallest=16 * 2880 * 2880,
             param="bf16", grad="bf16", packed=False),
        # many small parameters (norm weights, routers, biases), views of flat buffers at odd offsets, fp32
        dict(name="adamw_many_small", op="adamw", count=60, largest=368641, smallest=1, param="f32", grad="f32",
             packed=True),
        # the experts of the first case with 8-bit states
        dict(name="adamw8_share128", op="adamw8", count=2, largest=16 * 2880 * 5760, smallest=16 * 2880 * 2880,
             param="bf16", grad="bf16", packed=False),
        # dense parameters of a few layers, fp32 weights and bf16 gradients, 8-bit states, ragged lengths
        dict(name="adamw8_layers", op="adamw8", count=24, largest=4096 * 1027, smallest=2880, param="f32", grad="bf16",
             packed=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "rms", "rms_bwd", "adamw", "adamw8"])
    while True:
        if op in ("route", "route_bwd"):
            score, bias = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
            groups = rng.choice([1, 1, 2, 3, 4, 8, 16])
            E = groups * _log_int(rng, 4, 1024 // groups)
            top_groups = rng.randint(1, groups)
            k = _log_int(rng, 1, min(16, top_groups * (E // groups)))
            case = dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=k, score=score, bias=bias, groups=groups,
                        top_groups=top_groups, renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                        held=rng.choice(["f32", "bf16"]))
            ok = case["T"] * E <= 1 << 25
        elif op in ("rms", "rms_bwd"):
            dtype = rng.choice(["bf16", "bf16", "f32"])
            case = dict(op=op, T=_log_int(rng, 1, 16384), d=8 * _log_int(rng, 1, 2048), dtype=dtype,
                        wdtype=rng.choice([dtype, "f32"]), residual=rng.random() < 0.6)
            if op == "rms":
                case["int8"] = dtype == "bf16" and rng.random() < 0.5
            ok = case["T"] * case["d"] * _BYTES[dtype] <= 16384 * 7168 * 2
        else:
            smallest = _log_int(rng, 1, 1 << 20)
            case = dict(op=op, count=_log_int(rng, 1, 150), largest=_log_int(rng, smallest, 1 << 27),
                        smallest=smallest, param=rng.choice(["bf16", "f32"]), grad=rng.choice(["bf16", "f32"]),
                        packed=rng.random() < 0.5)
            ok = sum(_sizes(case)) <= 16 * 2880 * 8640 // 2
        if ok:
            return case


# --------------------------------------------------------------------- the work

def _sizes(case):
    """Element counts of the tensors: the largest, the smallest, the rest log-uniform between."""
    rng = random.Random(f"{case['count']}/{case['largest']}/{case['smallest']}")
    mid = [_log_int(rng, case["smallest"], case["largest"]) for _ in range(max(0, case["count"] - 2))]
    return [case["largest"]] + mid + ([case["smallest"]] if case["count"] > 1 else [])


def work(case):
    op = case["op"]
    if op == "route":  # logits read, ids and weights written
        T, E, k = case["T"], case["E"], case["k"]
        return dict(bytes=4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), flops=T * E * 6)
    if op == "route_bwd":  # ids, their weights' gradients and logits read, every logit's gradient written
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == "softmax" and not case["renormalize"]
        return dict(bytes=4 * T * E + 8 * T * k + 4 * T * (E if dense else k), flops=T * (E * 6 if dense else k * 10))
    if op == "rms":
        T, d, b = case["T"], case["d"], _BYTES[case["dtype"]]
        codes = T * 64 * ((d + 63) // 64) + 4 * T if case["int8"] else 0
        return dict(bytes=T * d * b * (4 if case["residual"] else 2) + codes + 4 * T + d * _BYTES[case["wdtype"]],
                    flops=T * d * (6 if case["int8"] else 5))
    if op == "rms_bwd":
        T, d, b = case["T"], case["d"], _BYTES[case["dtype"]]
        return dict(bytes=T * d * b * (4 if case["residual"] else 3) + 4 * T + 2 * d * _BYTES[case["wdtype"]],
                    flops=T * d * 10)
    n = sum(_sizes(case))
    params = 8 + 2 if case["param"] == "bf16" else 8  # the fp32 values read and written, a bf16 copy written
    states = 16 if op == "adamw" else 4
    scales = 0 if op == "adamw" else 16 * sum((s + _BLOCK - 1) // _BLOCK for s in _sizes(case))
    return dict(bytes=n * (_BYTES[case["grad"]] + params + states) + scales + 4, flops=n * 16)


# -------------------------------------------------------------------- the inputs

def _round_up(n, to):
    return (n + to - 1) // to * to


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1 + 7919 * seed)
    op = case["op"]

    def normal(shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev).mul_(std).add_(mean).to(dtype)

    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        # experts that are liked more than others, held as the router's product leaves them
        x = (normal((T, E)) + normal((E,), 0.5)).to(_DT[case["held"]]).float()
        st = dict(case=case, x=x, bias=normal((E,), 0.05) if case["bias"] else None)
        if op == "route_bwd":  # distinct experts of each token, likelier the larger their logit
            st["idx"] = torch.topk(x + normal((T, E), 0.1), k, dim=1).indices.to(torch.int32)
            st["dw"] = normal((T, k), 0.1)
        return st
    if op in ("rms", "rms_bwd"):
        T, d, dt, wdt = case["T"], case["d"], _DT[case["dtype"]], _DT[case["wdtype"]]
        # a residual stream's rows: a few large channels
        x = (normal((T, d)) * torch.exp(normal((d,), 0.5))).to(dt)
        st = dict(case=case, x=x, w=normal((d,), 0.2, 1.0, wdt))
        if op == "rms":
            st["r"] = normal((T, d), 0.5, 0.0, dt) if case["residual"] else None
        else:
            f = x.double()
            st["rstd"] = (1.0 / torch.sqrt((f * f).mean(dim=1) + _EPS)).float()
            st["dy"] = normal((T, d), 1.0, 0.0, dt)
            st["ds"] = normal((T, d), 1.0, 0.0, dt) if case["residual"] else None
        return st
    return _prepare_adamw(case, gen, dev)


def _prepare_adamw(case, gen, dev):
    """Flat buffers of weights, gradients and states, and the tensors as views of them:
    one after the other (packed), or each at a multiple of 128 elements."""
    eight, sizes = case["op"] == "adamw8", _sizes(case)

    def places(step):
        at = [0]
        for n in sizes:
            at.append(at[-1] + _round_up(n, step))
        return at

    plain = places(1 if case["packed"] else _BLOCK)
    held = places(_BLOCK) if eight else plain

    def fill(total, std):
        out = torch.empty(total, device=dev)
        for at in range(0, total, 1 << 27):
            part = out[at:at + (1 << 27)]
            part.copy_(torch.randn(part.numel(), generator=gen, device=dev)).mul_(std)
        return out

    # gradients of one parameter differ in size from element to element, and its states follow them
    p = fill(plain[-1], 0.02)
    g = fill(plain[-1], 1e-3)
    m = fill(held[-1], 3e-4)
    v = fill(held[-1], 1e-3).abs_().add_(1e-4)
    norm = torch.linalg.vector_norm(g).reshape(1)
    st = dict(case=case, at=plain, held=held, sizes=sizes, norm=norm, max_norm=0.8 * float(norm))
    st["p"] = p.to(_DT[case["param"]])
    st["master"] = p if case["param"] == "bf16" else None
    st["g"] = g.to(_DT[case["grad"]])
    if eight:
        st["m"], st["ms"] = _codes(m, False)
        st["v"], st["vs"] = _codes(v, True)
    else:
        st["m"], st["v"] = m, v.mul_(v)
    st["lists"] = _lists(st)
    return st


def _views(flat, at, sizes):
    return [flat[a:a + n] for a, n in zip(at, sizes)]


def _lists(st):
    """The lists that a user's program holds."""
    at, held, sizes = st["at"], st["held"], st["sizes"]
    lists = dict(params=_views(st["p"], at, sizes), grads=_views(st["g"], at, sizes), m=_views(st["m"], held, sizes),
                 v=_views(st["v"], held, sizes),
                 masters=None if st["master"] is None else _views(st["master"], at, sizes))
    if st["case"]["op"] == "adamw8":
        blocks = [(n + _BLOCK - 1) // _BLOCK for n in sizes]
        first = [a // _BLOCK for a in held]
        lists["ms"], lists["vs"] = _views(st["ms"], first, blocks), _views(st["vs"], first, blocks)
    return lists


def _codes(a, root):
    """e4m3 codes of a flat array of whole blocks and their scales."""
    b = a.reshape(-1, _BLOCK)
    scale = torch.clamp(b.abs().amax(dim=1) / 448.0, min=2.0 ** -126)
    q = (b * (1.0 / scale)[:, None]).to(torch.float8_e4m3fn)
    if root:
        q = torch.where((b > 0) & (q.float() == 0), torch.full_like(b, 2.0 ** -9), q.float()).to(torch.float8_e4m3fn)
    return q.reshape(-1), scale


# ------------------------------------------------------------------------ a pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own[op](state)
    return _plain[op](state)


def _scores(x, score):
    """Scores in 64 bits: the order of near ones hangs on them."""
    x = x.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    p = torch.exp(x - x.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _plain_route(st):
    c, x = st["case"], st["x"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    s = _scores(x, c["score"])
    by = x
    if st["bias"] is not None or G > 1:
        by = (s if st["bias"] is None else s + st["bias"].double()).float()
    if G > 1:
        best = torch.sort(by.reshape(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        mask[torch.arange(T, device=x.device)[:, None], kept] = True
        by = torch.where(mask[:, :, None].expand(T, G, E // G).reshape(T, E), by, torch.full_like(by, -math.inf))
    idx = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    w = s[torch.arange(T, device=x.device)[:, None], idx]
    if c["renormalize"]:
        w = w / (w.sum(dim=1, keepdim=True) + (1e-20 if c["score"] == "sigmoid" else 0.0))
    return [idx.to(torch.int32), (w * c["scale"]).float()]


def _plain_route_bwd(st):
    c, x = st["case"], st["x"]
    rows, idx, dw = torch.arange(c["T"], device=x.device)[:, None], st["idx"].long(), st["dw"] * c["scale"]
    dx = torch.zeros_like(x)
    if c["score"] == "sigmoid":
        xs = x[rows, idx]
        s = 1.0 / (1.0 + torch.exp(-xs))
        if c["renormalize"]:
            total = s.sum(dim=1, keepdim=True) + 1e-20
            dw = (dw - (dw * s).sum(dim=1, keepdim=True) / total) / total
        dx[rows, idx] = dw * s / (1.0 + torch.exp(xs))
    elif c["renormalize"]:
        xs = x[rows, idx]
        q = torch.exp(xs - xs.amax(dim=1, keepdim=True))
        q = q / q.sum(dim=1, keepdim=True)
        dx[rows, idx] = q * (dw - (dw * q).sum(dim=1, keepdim=True))
    else:
        p = torch.exp(x - x.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
        dx[rows, idx] = dw
        dx = p * (dx - (dw * p[rows, idx]).sum(dim=1, keepdim=True))
    return dx


def _plain_rms(st):
    x = st["x"]
    s = x if st["r"] is None else (x.float() + st["r"].float()).to(x.dtype)
    f = s.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(dim=1) + _EPS)
    y = f * rstd[:, None] * st["w"].float()
    out = [y.to(x.dtype), s, rstd]
    if st["case"]["int8"]:
        T, d = x.shape
        scale = torch.clamp(y.abs().amax(dim=1) / 127.0, min=2.0 ** -126)
        q = torch.zeros((T, _round_up(d, 64)), device=x.device)
        q[:, :d] = torch.round(y * (1.0 / scale)[:, None])
        q = q.reshape(T, -1, 64).permute(1, 0, 2).contiguous().to(torch.int8)
        out += [_values(q, scale), scale]
    return out


def _values(q, scale):
    """What 8-bit rows [ceil(d / 64), T, 64] stand for."""
    return torch.mul(q, scale[None, :, None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))


def _plain_rms_bwd(st):
    dy = st["dy"].float()
    h = st["x"].float() * st["rstd"][:, None]
    g = dy * st["w"].float()
    dx = st["rstd"][:, None] * (g - h * (g * h).mean(dim=1, keepdim=True))
    if st["ds"] is not None:
        dx = dx + st["ds"].float()
    return [dx.to(st["x"].dtype), (dy * h).sum(dim=0).to(st["w"].dtype)]


def _adamw_step(p, g, m, v, coef):
    """(p, m, v) after a step on fp32 values."""
    g = g.float() * coef
    m = m * _B1 + g * (1.0 - _B1)
    v = v * _B2 + g * g * (1.0 - _B2)
    p = p * (1.0 - _LR * _WD)
    root = torch.sqrt(v)
    p = p - (_LR / (1.0 - _B1 ** _STEP)) * (m / (root * (1.0 / math.sqrt(1.0 - _B2 ** _STEP)) + _AEPS))
    return p, m, v, root


def _plain_adamw(st):
    coef = torch.clamp(st["max_norm"] / (st["norm"] + 1e-6), max=1.0)
    lists = st["lists"]
    masters = lists["masters"] or lists["params"]
    for p, w, g, m, v in zip(lists["params"], masters, lists["grads"], lists["m"], lists["v"]):
        new, m2, v2, _ = _adamw_step(w, g, m, v, coef)
        m.copy_(m2)
        v.copy_(v2)
        w.copy_(new)
        if w is not p:
            p.copy_(new.to(p.dtype))
    return _adamw_out(st)


def _plain_adamw8(st):
    coef = torch.clamp(st["max_norm"] / (st["norm"] + 1e-6), max=1.0)
    lists = st["lists"]
    masters = lists["masters"] or lists["params"]
    for p, w, g, m, ms, v, vs in zip(lists["params"], masters, lists["grads"], lists["m"], lists["ms"], lists["v"],
                                     lists["vs"]):
        n = p.numel()
        rows = torch.arange(n, device=p.device) // _BLOCK
        root = v.float() * vs[rows]
        new, m2, _, root = _adamw_step(w, g, m.float() * ms[rows], root * root, coef)
        for a, codes, scale, is_root in ((m2, m, ms, False), (root, v, vs, True)):
            whole = torch.zeros(scale.numel() * _BLOCK, device=p.device)
            whole[:n] = a
            q, sc = _codes(whole, is_root)
            codes.view(torch.uint8).copy_(q[:n].view(torch.uint8))
            scale.copy_(sc)
        w.copy_(new)
        if w is not p:
            p.copy_(new.to(p.dtype))
    return _adamw_out(st)


def _adamw_out(st):
    keys = ("p", "master", "m", "v") + (("ms", "vs") if st["case"]["op"] == "adamw8" else ())
    return [st[k] for k in keys if st[k] is not None]


_plain = dict(route=_plain_route, route_bwd=_plain_route_bwd, rms=_plain_rms, rms_bwd=_plain_rms_bwd,
              adamw=_plain_adamw, adamw8=_plain_adamw8)


def _router(st):
    import token_dispatch_grouped_amd as moe
    c = st["case"]
    return moe.Router(score=c["score"], bias=st["bias"], groups=c["groups"], top_groups=c["top_groups"],
                      group_score="top2", renormalize=c["renormalize"], scale=c["scale"])


def _own_route(st):
    import token_dispatch_grouped_amd as moe
    idx, w = moe.route_experts(st["x"], st["case"]["k"], _router(st))
    return [idx, w]


def _own_route_bwd(st):
    import token_dispatch_grouped_amd as moe
    return moe.route_experts_backward(st["x"], st["idx"], st["dw"], _router(st))


def _own_rms(st):
    import token_dispatch_grouped_amd as moe
    if st["case"]["int8"]:
        rows, y, s, rstd = moe.rms_norm_int8(st["x"], st["w"], _EPS, residual=st["r"])
        return [y, s, rstd, _values(rows.codes, rows.scale), rows.scale]
    y, s, rstd = moe.rms_norm(st["x"], st["w"], _EPS, residual=st["r"])
    return [y, s, rstd]


def _own_rms_bwd(st):
    import token_dispatch_grouped_amd as moe
    dx, dw = moe.rms_norm_backward(st["dy"], st["x"], st["w"], st["rstd"], d_s=st["ds"])
    return [dx, dw]


def _own_adamw(st):
    import token_dispatch_grouped_amd as moe
    li = st["lists"]
    m, v = li["m"], li["v"]
    if st["case"]["op"] == "adamw8":
        m = [moe.Float8State(c, s) for c, s in zip(m, li["ms"])]
        v = [moe.Float8State(c, s) for c, s in zip(v, li["vs"])]
    moe.adamw(li["params"], li["grads"], m, v, step=_STEP, lr=_LR, betas=(_B1, _B2), eps=_AEPS, weight_decay=_WD,
              masters=li["masters"], norm=st["norm"], max_norm=st["max_norm"])
    return _adamw_out(st)


_own = dict(route=_own_route, route_bwd=_own_route_bwd, rms=_own_rms, rms_bwd=_own_rms_bwd, adamw=_own_adamw,
            adamw8=_own_adamw)


# ------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "route_bwd":
        # w as a function of the logits, differentiated by the product rule written out as a matrix
        x, idx, up = st["x"].double(), st["idx"].long(), st["dw"].double() * case["scale"]
        out = torch.zeros_like(x)
        if case["score"] == "softmax" and not case["renormalize"]:
            p = torch.softmax(x, dim=1)
            picked = torch.gather(p, 1, idx)
            out -= p * (up * picked).sum(dim=1, keepdim=True)
            return out.scatter_add_(1, idx, up * picked)
        z = torch.gather(x, 1, idx)
        if case["score"] == "softmax":
            q = torch.softmax(z, dim=1)
            jac = torch.diag_embed(q) - q[:, :, None] * q[:, None, :]
        else:
            s = torch.sigmoid(z)
            slope = s * torch.sigmoid(-z)
            if case["renormalize"]:
                total = s.sum(dim=1)[:, None, None] + 1e-20
                jac = torch.diag_embed(slope) / total - s[:, :, None] * slope[:, None, :] / total ** 2
            else:
                jac = torch.diag_embed(slope)
        return out.scatter_(1, idx, (up[:, :, None] * jac).sum(dim=1))
    if op == "rms":
        s = st["x"].double()
        if st["r"] is not None:  # the sum is held in x's type: the rest of the operator starts from it
            s = (s + st["r"].double()).to(st["x"].dtype).double()
        rstd = torch.rsqrt(torch.linalg.vector_norm(s, dim=1) ** 2 / case["d"] + _EPS)
        y = s * st["w"].double() * rstd.unsqueeze(1)
        out = [y, s, rstd]
        if case["int8"]:
            step = torch.clamp_min(torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127, 2.0 ** -126)
            v = torch.round(y / step.unsqueeze(1)) * step.unsqueeze(1)
            v = torch.nn.functional.pad(v, (0, -case["d"] % 64)).unflatten(1, (-1, 64)).transpose(0, 1).contiguous()
            out += [v, step]
        return out
    if op == "rms_bwd":
        dy, w, rstd = st["dy"].double(), st["w"].double(), st["rstd"].double().unsqueeze(1)
        h = st["x"].double() * rstd
        dot = torch.mv(dy * h, w).unsqueeze(1) / case["d"]
        dx = (dy * w - h * dot) * rstd
        if st["ds"] is not None:
            dx += st["ds"].double()
        return [dx, torch.multiply(dy, h, out=h).sum(dim=0)]
    return _exact_adamw(case, st)


def _exact_route(case, st):
    x = st["x"].double()
    T, E, k, G, P = case["T"], case["E"], case["k"], case["groups"], case["top_groups"]
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, dim=1)
    choice = x
    if case["bias"] or G > 1:  # what the choice goes by is held in 32 bits
        choice = (s + (st["bias"].double() if case["bias"] else 0.0)).to(torch.float32).double()
    if G > 1:
        two = torch.topk(choice.unflatten(1, (G, E // G)), 2, dim=2).values.to(torch.float32)
        best = (two[:, :, 0] + two[:, :, 1]).double()
        # a group's place: how many others are before it
        lower = torch.arange(G, device=x.device)[:, None] > torch.arange(G, device=x.device)[None, :]
        ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & lower)
        choice = choice.masked_fill((ahead.sum(dim=2) >= P).repeat_interleave(E // G, dim=1), -math.inf)
    idx = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :k]
    w = torch.gather(s, 1, idx)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return [idx.to(torch.int32), w * case["scale"]]


def _e4m3(a):
    """The nearest e4m3 value (ties to even) of values of at most 448, in 64 bits."""
    exponent = torch.clamp_min(torch.frexp(a).exponent - 1, -6)
    ulp = torch.ldexp(torch.ones_like(a), exponent - 3)
    return torch.round(a / ulp) * ulp


def _exact_adamw(case, st):
    eight, li = case["op"] == "adamw8", st["lists"]
    coef = min(1.0, st["max_norm"] / (float(st["norm"]) + 1e-6))
    flat = {k: st[k].to(torch.float64) for k in ("p", "master", "m", "v") if st[k] is not None}
    if eight:
        flat["ms"], flat["vs"] = st["ms"].double(), st["vs"].double()
    chunk = 1 << 24
    for i, n in enumerate(st["sizes"]):
        for lo in range(0, n, chunk):
            hi = min(n, lo + chunk)
            here = slice(st["at"][i] + lo, st["at"][i] + hi)
            there = slice(st["held"][i] + lo, st["held"][i] + hi)
            blocks = slice(there.start // _BLOCK, (there.stop + _BLOCK - 1) // _BLOCK)
            g = li["grads"][i][lo:hi].double() * coef
            m, v = flat["m"][there], flat["v"][there]
            if eight:
                times = lambda s: s[blocks].repeat_interleave(_BLOCK)[:hi - lo]  # noqa: E731
                m, v = m * times(flat["ms"]), (v * times(flat["vs"])) ** 2
            m = torch.lerp(g, m, torch.full_like(m, _B1))
            v = torch.lerp(g * g, v, torch.full_like(v, _B2))
            p = flat["p" if st["master"] is None else "master"][here]
            hat = m / (1 - _B1 ** _STEP) / (torch.sqrt(v / (1 - _B2 ** _STEP)) + _AEPS)
            p = p - _LR * (_WD * p + hat)
            for k in ("p", "master"):
                if k in flat:
                    flat[k][here] = p
            if eight:
                for k, scales, a in (("m", "ms", m), ("v", "vs", torch.sqrt(v))):
                    whole = torch.nn.functional.pad(a, (0, -(hi - lo) % _BLOCK)).unflatten(0, (-1, _BLOCK))
                    step = torch.clamp_min(whole.abs().max(dim=1).values / 448, 2.0 ** -126)
                    q = _e4m3(whole / step.unsqueeze(1))
                    if k == "v":
                        q = torch.where((whole > 0) & (q == 0), 2.0 ** -9, q)
                    flat[k][there] = q.flatten()[:hi - lo]
                    flat[scales][blocks] = step
            else:
                flat["m"][there], flat["v"][there] = m, v
    keys = ("p", "master", "m", "v") + (("ms", "vs") if eight else ())
    return [flat[k] for k in keys if k in flat]
