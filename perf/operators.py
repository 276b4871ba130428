"""The gated linear recurrence and the gradient-clipping operators as a user's
program calls them, their plain forms and their definitions in 64 bits.

Operators
  scan   h_t = a_t h_{t-1} + x_t (coupled: a_t h_{t-1} + (1 - a_t) x_t) along
         every sequence; all states and the last one of each sequence
  train  the same, and the gradients w.r.t. gates, inputs and first states
  rays   compositing of ray samples: the coupled recurrence, back to front,
         one gate per sample for all its colour channels, last state only,
         and its gradients
  step   one token of the recurrence for a batch of kept states
  clip   2-norm over a list of gradient tensors, and the scaled gradients
  adam   the same norm, and the Adam step on the scaled gradients
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ES = {"f32": 4, "bf16": 2, "f16": 2}
CLIP_EPS = 1e-6
LR = {"means": 1.6e-4, "log_scales": 5e-3, "quats": 1e-3, "logit_opacity": 5e-2, "colors": 2.5e-3}
BETA1, BETA2, EPS, STEP, WARMUP = 0.9, 0.999, 1e-15, 10, 3000
GROUPS = ("means", "log_scales", "quats", "logit_opacity", "colors")
GRADS = ("dL_dmeans", "dL_dscales", "dL_dquats", "dL_dopacity", "dL_dcolors")


def _scan(name, op, S, T, C, G, x, a, ragged, reverse, coupled, h0):
    c = {"op": op, "S": S, "T": T, "C": C, "G": G, "x": x, "a": a, "ragged": ragged, "reverse": reverse,
         "coupled": coupled, "h0": h0}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one long sequence of few channels, fp32: nothing but the time axis to split
        _scan("scan-long-f32", "scan", 1, 131072, 64, 64, "f32", "f32", False, False, False, False),
        # a packed batch of ragged sequences, 16-bit states with one fp32 gate per head of 64 channels
        _scan("scan-packed-heads-bf16", "scan", 48, 24576, 640, 10, "bf16", "f32", True, False, False, True),
        # a small training batch of odd sizes
        _scan("train-odd-f16", "train", 5, 5 * 1237, 333, 333, "f16", "f16", False, False, False, True),
        # a layer's training step at full size
        _scan("train-large-bf16", "train", 8, 8 * 8192, 2048, 2048, "bf16", "bf16", False, False, False, False),
        # the samples of a 64 x 64 image's rays
        _scan("rays-64px", "rays", 64 * 64, 98304, 3, 1, "f32", "f32", True, True, True, True),
        # the samples of an 800 x 800 image's rays
        _scan("rays-800px", "rays", 800 * 800, 24000007, 3, 1, "f32", "f32", True, True, True, True),
        # one token of one sequence
        {"name": "step-one", "op": "step", "S": 1, "C": 256, "G": 256, "x": "f32", "a": "f32", "coupled": False},
        # one token of a full serving batch, 16-bit tokens and fp32 states
        {"name": "step-batch", "op": "step", "S": 4096, "C": 2048, "G": 2048, "x": "bf16", "a": "f32",
         "coupled": False},
        # the gradients of a scene of 10,000 Gaussians (RGB)
        {"name": "clip-scene-10k", "op": "clip", "sizes": "scene", "N": 10000, "K": 3, "tight": True},
        # the gradients of a large model: 148 tensors from 1 element up, fp32 and bf16 mixed
        {"name": "clip-many", "op": "clip", "sizes": "many", "N": 200000000, "K": 148, "tight": True},
        # the optimiser step of 10,000 Gaussians (RGB)
        {"name": "adam-10k", "op": "adam", "N": 10000, "K": 3, "tight": True},
        # the optimiser step of 1,000,000 Gaussians with spherical harmonics of degree 3
        {"name": "adam-1M-sh3", "op": "adam", "N": 1000000, "K": 48, "tight": True},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "rays", "step", "clip", "adam"])
    tight = rng.random() < 0.7
    if op in ("scan", "train"):
        x = rng.choice(["f32", "bf16", "f16"])
        per_head = rng.choice([1, 1, 1, 2, 5, 16, 64, 128])
        G = _logint(rng, 1, 2048 // per_head)
        C = G * per_head
        ragged = rng.random() < 0.5
        rows = _logint(rng, 1, min(200000, 40000000 // C))
        S = _logint(rng, 1, max(1, min(rows, 256)))
        T = rows if ragged else max(1, rows // S) * S
        return _scan(None, op, S, T, C, G, x, rng.choice([x, "f32"]), ragged, rng.random() < 0.3,
                     rng.random() < 0.3, rng.random() < 0.5)
    if op == "rays":
        S = _logint(rng, 1, 500000)
        return _scan(None, op, S, int(S * rng.uniform(1.0, 40.0)), rng.choice([1, 3, 4, 7]), 1, "f32", "f32", True,
                     rng.random() < 0.7, True, True)
    if op == "step":
        C = _logint(rng, 1, 4096)
        x = rng.choice(["f32", "bf16", "f16"])
        return {"op": "step", "S": _logint(rng, 1, max(1, 8000000 // C)), "C": C, "G": rng.choice([1, C]), "x": x,
                "a": rng.choice([x, "f32"]), "coupled": rng.random() < 0.3}
    if op == "clip":
        if rng.random() < 0.5:
            return {"op": "clip", "sizes": "scene", "N": _logint(rng, 1, 3000000), "K": rng.choice([3, 12, 48]),
                    "tight": tight}
        return {"op": "clip", "sizes": "many", "N": _logint(rng, 1000, 100000000), "K": _logint(rng, 1, 600),
                "tight": tight}
    return {"op": "adam", "N": _logint(rng, 1, 900000), "K": rng.choice([3, 12, 27, 48]), "tight": tight}


# ---- inputs -------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _scan_inputs(case, seed):
    g = _gen(seed)
    S, T, C, G = case["S"], case["T"], case["C"], case["G"]
    d = {}
    if case["ragged"]:  # cut points at random: lengths from 0 up, ragged as packed batches and rays are
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values
        d["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
        shape = (T,)
    else:
        d["offsets"] = None
        shape = (S, T // S)
    if case["op"] == "rays":  # transmittances exp(-density * length), half of the samples in empty space
        d["a"] = torch.exp(-0.2 * torch.relu(_randn(g, *shape, G)))
        d["x"] = torch.rand((*shape, C), generator=g, device="cuda")
        d["h0"] = torch.rand((S, C), generator=g, device="cuda")  # background
    else:  # forget gates, most of them close to 1
        d["a"] = torch.sigmoid(3.0 + 1.5 * _randn(g, *shape, G))
        d["x"] = _randn(g, *shape, C)
        d["h0"] = _randn(g, S, C) if case["h0"] else None
    d["a"] = d["a"].to(DT[case["a"]])
    d["x"] = d["x"].to(DT[case["x"]])
    if case["op"] != "scan":
        d["dh"] = _randn(g, *shape, C).to(DT[case["x"]]) if case["op"] == "train" else None
        d["dh_last"] = _randn(g, S, C)
    return d


def _step_inputs(case, seed):
    g = _gen(seed)
    S, C, G = case["S"], case["C"], case["G"]
    return {"a": torch.sigmoid(3.0 + 1.5 * _randn(g, S, G)).to(DT[case["a"]]), "x": _randn(g, S, C).to(DT[case["x"]]),
            "state": _randn(g, S, C)}


def _scene_shapes(N, C):
    return [(N, 3), (N, 3), (N, 4), (N,), (N, C)]


def _many_sizes(case):
    """Sizes of K tensors, N elements in all: vectors from 1 element up and
    matrices thousands of times larger, in an order that mixes them."""
    K, N = case["K"], case["N"]
    w = [math.exp(9.0 * ((i * 0.6180339887) % 1.0)) for i in range(K)]
    s = sum(w)
    return [max(1, int(N * v / s)) for v in w]


def _clip_inputs(case, seed):
    g = _gen(seed)
    if case["sizes"] == "scene":
        return [_randn(g, *s) * 10.0 ** (-1 - i % 3) for i, s in enumerate(_scene_shapes(case["N"], case["K"]))]
    return [(_randn(g, n) * 10.0 ** (-1 - i % 3)).to(torch.float32 if i % 4 == 0 else torch.bfloat16)
            for i, n in enumerate(_many_sizes(case))]


def _buckets(tensors, make):
    """One flat buffer per type, filled by `make`, and the tensors' places in
    it (each on a boundary of 64 elements), as gradient buckets are kept."""
    used, places = {}, []
    for t in tensors:
        o = used.get(t.dtype, 0)
        places.append((t.dtype, o, t.numel(), t.shape))
        used[t.dtype] = o + (t.numel() + 63) // 64 * 64
    flat = {dt: make(n, dt) for dt, n in used.items()}
    return list(flat.values()), [flat[dt][o:o + n].view(shape) for dt, o, n, shape in places]


def _max_norm(case, total):
    """Clipping bound: below the expected norm ("tight"), or a hundred times that."""
    return 0.02 * math.sqrt(total) * (1.0 if case["tight"] else 100.0)


def _adam_inputs(case, seed):
    g = _gen(seed)
    N, C = case["N"], case["K"]
    sh = _scene_shapes(N, C)
    d = {"params": {"means": 2.0 * _randn(g, N, 3), "log_scales": -4.5 + 0.7 * _randn(g, N, 3),
                    "quats": torch.nn.functional.normalize(_randn(g, N, 4), dim=1),
                    "logit_opacity": 1.5 * _randn(g, N), "colors": _randn(g, N, C)},
         "grads": {k: _randn(g, *s) * (10.0 if k == "dL_dscales" else 0.1) for k, s in zip(GRADS, sh)}}
    d["m"] = 0.05 * _randn(g, (11 + C) * N)
    d["v"] = torch.square(0.05 * _randn(g, (11 + C) * N)) + 1e-4
    return d


def _total(case):
    if case["op"] == "adam" or case["sizes"] == "scene":
        return case["N"] * (11 + case["K"])
    return sum(_many_sizes(case))


def prepare(case, seed):
    op = case["op"]
    if op in ("scan", "train", "rays"):
        st = _scan_inputs(case, seed)
        if op != "scan":
            for k in ("a", "x", "h0"):
                if st[k] is not None:
                    st[k].requires_grad_(True)
        if own:
            from differentiable_gaussian_splatting_preprocess_b200 import autograd as GA
            st["ws"] = GA.scan_workspace(st["a"], st["x"], seq_offsets=st["offsets"])
        else:
            o = st["offsets"]
            st["longest"] = case["T"] // case["S"] if o is None else int((o[1:] - o[:-1]).max())
    elif op == "step":
        st = _step_inputs(case, seed)
        st["next"] = torch.empty_like(st["state"])
    elif op == "clip":
        st = {"grads": _clip_inputs(case, seed), "max_norm": _max_norm(case, _total(case))}
        st["flat"], st["out"] = _buckets(st["grads"], lambda n, dt: torch.zeros(n, dtype=dt, device="cuda"))
        if own:
            from differentiable_gaussian_splatting_preprocess_b200 import optim
            st["list"] = optim.GradList(st["grads"])
            st["out_list"] = optim.GradList(st["out"])
    else:
        st = _adam_inputs(case, seed)
        N = case["N"]
        st["max_norm"] = _max_norm(case, _total(case))
        st["scales"] = torch.empty((N, 3), device="cuda")
        st["opacity"] = torch.empty((N,), device="cuda")
        if own:
            from differentiable_gaussian_splatting_preprocess_b200 import binding as B
            from differentiable_gaussian_splatting_preprocess_b200 import optim
            st["cfg"] = B.GsAdamConfig(LR["means"], LR["log_scales"], LR["quats"], LR["logit_opacity"], LR["colors"],
                                       BETA1, BETA2, EPS, WARMUP)
            st["list"] = optim.GradList([st["grads"][k] for k in GRADS])
    st["case"] = case
    return st


# ---- one pass -----------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    case = st["case"]
    op = case["op"]
    if op in ("scan", "train", "rays"):
        from differentiable_gaussian_splatting_preprocess_b200 import autograd as GA
        h, last = GA.gated_scan(st["a"], st["x"], h0=st["h0"], seq_offsets=st["offsets"], reverse=case["reverse"],
                                coupled=case["coupled"], final_only=op == "rays", workspace=st["ws"])
        if op == "scan":
            return {"h": h, "h_last": last}
        ins = [st["a"], st["x"]] + ([st["h0"]] if st["h0"] is not None else [])
        outs, gs = ([h, last], [st["dh"], st["dh_last"]]) if h is not None else ([last], [st["dh_last"]])
        grads = torch.autograd.grad(outs, ins, gs)
        r = {"h_last": last.detach(), "da": grads[0], "dx": grads[1]}
        if h is not None:
            r["h"] = h.detach()
        if len(grads) > 2:
            r["dh0"] = grads[2]
        return r
    if op == "step":
        from differentiable_gaussian_splatting_preprocess_b200 import autograd as GA
        h, s = GA.scan_step(st["a"], st["x"], st["state"], out_state=st["next"], coupled=case["coupled"])
        return {"h": h, "state": s}
    from differentiable_gaussian_splatting_preprocess_b200 import optim
    if op == "clip":
        norm = optim.clip_grads(st["list"], st["max_norm"], out=st["out_list"])
        return {"norm": norm, "grads": st["flat"]}
    from differentiable_gaussian_splatting_preprocess_b200 import binding as B
    norm = optim.grad_norm(st["list"])
    B.gs_adam_step_clipped(st["cfg"], STEP, st["params"], st["grads"], st["m"], st["v"], norm, st["max_norm"],
                           st["scales"], st["opacity"])
    return {"norm": norm, "params": st["params"], "m": st["m"], "v": st["v"], "scales": st["scales"],
            "opacity": st["opacity"]}


def _doubling(a, b, pos, longest):
    """Inclusive scan of h_t = a_t h_{t-1} + b_t over rows: after the step of
    width d, (a, b) of a row stand for the last 2 d rows of its sequence."""
    d = 1
    while d < longest:
        inside = (pos[d:] >= d)[:, None, None]
        nb = b.clone()
        nb[d:] += torch.where(inside, a[d:] * b[:-d], torch.zeros((), device=b.device))
        na = a.clone()
        na[d:] = torch.where(inside, a[d:] * a[:-d], a[d:])
        a, b = na, nb
        d *= 2
    return b


def _plain_scan(st):
    case = st["case"]
    S, T, C, G = case["S"], case["T"], case["C"], case["G"]
    rev, cpl, longest = case["reverse"], case["coupled"], st["longest"]
    a = st["a"].detach().float().reshape(T, G, 1)
    x = st["x"].detach().float().reshape(T, G, C // G)
    h0 = (st["h0"].detach() if st["h0"] is not None else torch.zeros((S, C), device=a.device)).reshape(S, G, C // G)
    rows = torch.arange(T, device=a.device)
    if st["offsets"] is None:
        off = torch.arange(S + 1, device=a.device) * (T // S)
    else:
        off = st["offsets"]
    seq = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    full = off[1:] > off[:-1]
    first, last = off[:-1], off[1:] - 1
    pos_f, pos_r = rows - off[seq], off[seq + 1] - 1 - rows
    if rev:
        first, last, pos_f, pos_r = last, first, pos_r, pos_f
    flip = (lambda t: torch.flip(t, (0,))) if rev else (lambda t: t)
    b = (1 - a) * x if cpl else x.clone()
    b[first[full]] += a[first[full]] * h0[full]
    h = flip(_doubling(flip(a), flip(b), flip(pos_f), longest))
    h_last = h0.clone()
    h_last[full] = h[last[full]]
    out = {"h_last": h_last.reshape(S, C)}
    shape = tuple(st["x"].shape)
    if case["op"] != "rays":
        out["h"] = h.reshape(shape).to(st["x"].dtype)
    if case["op"] == "scan":
        return out
    # adjoint: g_t = dh_t + a_{t+1} g_{t+1}
    dl = st["dh_last"].reshape(S, G, C // G)
    g = st["dh"].float().reshape(T, G, C // G).clone() if st["dh"] is not None else torch.zeros_like(x)
    g[last[full]] += dl[full]
    an = torch.zeros_like(a)  # the gate of the next row in scan order
    prev = torch.zeros_like(h)  # the state before the row
    if rev:
        an[1:], prev[:-1] = a[:-1], h[1:]
    else:
        an[:-1], prev[1:] = a[1:], h[:-1]
    an[last[full]] = 0
    prev[first[full]] = h0[full]
    g = flip(torch.flip(_doubling(torch.flip(flip(an), (0,)), torch.flip(flip(g), (0,)),
                                  torch.flip(flip(pos_r), (0,)), longest), (0,)))
    da = (g * (prev - x if cpl else prev)).sum(2)
    dx = (1 - a) * g if cpl else g
    out["da"] = da.reshape(st["a"].shape).to(st["a"].dtype)
    out["dx"] = dx.reshape(shape).to(st["x"].dtype)
    if st["h0"] is not None:
        dh0 = dl.clone()
        dh0[full] = a[first[full]] * g[first[full]]
        out["dh0"] = dh0.reshape(S, C)
    return out


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op in ("scan", "train", "rays"):
        with torch.no_grad():
            return _plain_scan(st)
    if op == "step":
        S, C, G = case["S"], case["C"], case["G"]
        a = st["a"].float().reshape(S, G, 1)
        x = st["x"].float().reshape(S, G, C // G)
        s = a * st["state"].reshape(S, G, C // G) + ((1 - a) * x if case["coupled"] else x)
        s = s.reshape(S, C)
        return {"h": s.to(st["x"].dtype), "state": s}
    if op == "clip":
        norm = torch.sqrt(sum(torch.sum(torch.square(t.double())) for t in st["grads"])).float()
        coef = torch.clamp(st["max_norm"] / (norm + CLIP_EPS), max=1.0)
        for t, o in zip(st["grads"], st["out"]):
            o.copy_((t.float() * coef).to(t.dtype))
        return {"norm": norm.reshape(1), "grads": st["flat"]}
    g = st["grads"]
    norm = torch.sqrt(sum(torch.sum(torch.square(g[k].double())) for k in GRADS)).float()
    coef = torch.clamp(st["max_norm"] / (norm + CLIP_EPS), max=1.0)
    p, N, off = st["params"], case["N"], 0
    for k, gk in zip(GROUPS, GRADS):
        gr = g[gk] * coef
        if k == "log_scales":
            gr = gr * torch.exp(p[k])
        elif k == "logit_opacity":
            o = 1 / (1 + torch.exp(-p[k]))
            gr = gr * o * (1 - o)
        n = gr.numel()
        m, v = st["m"][off:off + n].view(gr.shape), st["v"][off:off + n].view(gr.shape)
        off += n
        m.mul_(BETA1).add_((1 - BETA1) * gr)
        v.mul_(BETA2).add_((1 - BETA2) * gr * gr)
        rate = LR[k] * (STEP / WARMUP if k in ("means", "log_scales") else 1.0)
        p[k].sub_(rate * (m / (1 - BETA1 ** STEP)) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS))
        if k == "quats":
            p[k].div_(torch.sqrt(torch.sum(p[k] * p[k], 1, keepdim=True)))
    torch.exp(p["log_scales"], out=st["scales"])
    torch.div(1.0, 1 + torch.exp(-p["logit_opacity"]), out=st["opacity"])
    return {"norm": norm.reshape(1), "params": p, "m": st["m"], "v": st["v"], "scales": st["scales"],
            "opacity": st["opacity"]}


# ---- work and exact values ----------------------------------------------

def work(case):
    op = case["op"]
    if op in ("scan", "train", "rays"):
        S, T, C, G = case["S"], case["T"], case["C"], case["G"]
        xs, gs, ss = T * C * ES[case["x"]], T * G * ES[case["a"]], S * C * 4
        nbytes = xs + gs + ss * (2 if case["h0"] else 1) + (0 if op == "rays" else xs)
        flops = T * C * (4 if case["coupled"] else 2)
        if op != "scan":
            nbytes += xs + gs + ss * (2 if case["h0"] else 1) + (xs if op == "train" else 0)
            flops += T * C * (8 if case["coupled"] else 6)
        if case["ragged"]:
            nbytes += 8 * (S + 1)
        return {"bytes": nbytes, "flops": flops}
    if op == "step":
        S, C, G = case["S"], case["C"], case["G"]
        return {"bytes": S * (2 * C * ES[case["x"]] + G * ES[case["a"]] + 8 * C), "flops": 2 * S * C}
    if op == "clip":
        if case["sizes"] == "scene":
            nbytes = 4 * _total(case)
        else:
            nbytes = sum(n * (4 if i % 4 == 0 else 2) for i, n in enumerate(_many_sizes(case)))
        return {"bytes": 2 * nbytes + 4, "flops": 3 * _total(case)}
    n = _total(case)
    return {"bytes": 4 * n * 7 + 16 * case["N"] + 4, "flops": 16 * n}


def _exact_scan(case, seed):
    d = _scan_inputs(case, seed)
    S, T, C, G = case["S"], case["T"], case["C"], case["G"]
    if d["offsets"] is None:
        beg = [i * (T // S) for i in range(S)]
        end = [b + T // S for b in beg]
    else:
        o = d["offsets"].tolist()
        beg, end = o[:-1], o[1:]
    beg, end = torch.tensor(beg, device="cuda"), torch.tensor(end, device="cuda")
    order = torch.argsort(end - beg, descending=True)
    beg, end = beg[order], end[order]
    lens = (end - beg).cpu()
    longest = int(lens[0])
    if longest > 150000:
        return None
    # the sequences sorted by length: those that still run at position t come first
    live = (S - torch.searchsorted(torch.flip(lens, (0,)).contiguous(), torch.arange(longest), right=True)).tolist()
    a = d["a"].double().reshape(T, G)
    x = d["x"].double().reshape(T, C)
    per = C // G
    wide = (lambda t: t) if per == 1 else (lambda t: t.repeat_interleave(per, dim=1))
    h0 = (d["h0"].double() if d["h0"] is not None else torch.zeros((S, C), dtype=torch.float64, device="cuda"))
    sgn, base = (-1, end - 1) if case["reverse"] else (1, beg)
    s = h0[order].clone()
    h = torch.zeros((T, C), dtype=torch.float64, device="cuda")
    before = torch.zeros((T, C), dtype=torch.float64, device="cuda") if case["op"] != "scan" else None
    for t in range(longest):
        n = live[t]
        i = base[:n] + sgn * t
        at, xt = wide(a[i]), x[i]
        if before is not None:
            before[i] = s[:n]
        s[:n] = at * s[:n] + ((1.0 - at) * xt if case["coupled"] else xt)
        h[i] = s[:n]
    back = torch.empty_like(order)
    back[order] = torch.arange(S, device="cuda")
    out = {"h_last": s[back]}
    shape = tuple(d["x"].shape)
    if case["op"] != "rays":
        out["h"] = h.reshape(shape)
    if case["op"] == "scan":
        return out
    del h
    k = d["dh_last"].double()[order].clone()  # what a row's state receives from the rows after it
    da = torch.zeros((T, G), dtype=torch.float64, device="cuda")
    dx = torch.zeros((T, C), dtype=torch.float64, device="cuda")
    dh = d["dh"].double().reshape(T, C) if d["dh"] is not None else None
    for t in range(longest - 1, -1, -1):
        n = live[t]
        i = base[:n] + sgn * t
        at = wide(a[i])
        gt = k[:n] + dh[i] if dh is not None else k[:n].clone()
        dat = gt * (before[i] - x[i]) if case["coupled"] else gt * before[i]
        da[i] = dat.reshape(n, G, per).sum(2)
        dx[i] = (1.0 - at) * gt if case["coupled"] else gt
        k[:n] = at * gt
    out["da"] = da.reshape(d["a"].shape)
    out["dx"] = dx.reshape(shape)
    if d["h0"] is not None:
        out["dh0"] = k[back]
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("scan", "train", "rays"):
        return _exact_scan(case, seed)
    if op == "step":
        d = _step_inputs(case, seed)
        a = d["a"].double().expand(case["S"], case["C"]) if case["G"] == 1 else d["a"].double()
        u = d["x"].double()
        h = torch.addcmul(u - a * u if case["coupled"] else u, a, d["state"].double())
        return {"h": h, "state": h}
    if op == "clip":
        grads = _clip_inputs(case, seed)
        norm = math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))
        c = min(1.0, _max_norm(case, _total(case)) / (norm + CLIP_EPS))
        flat, places = _buckets(grads, lambda n, dt: torch.zeros(n, dtype=torch.float64, device="cuda"))
        for t, o in zip(grads, places):
            o.copy_(t.double() * c)
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "grads": flat}
    d = _adam_inputs(case, seed)
    gs = [d["grads"][k].double() for k in GRADS]
    norm = math.sqrt(math.fsum(float((t * t).sum()) for t in gs))
    c = min(1.0, _max_norm(case, _total(case)) / (norm + CLIP_EPS))
    params = {k: t.double() for k, t in d["params"].items()}
    gs[1] = gs[1] * params["log_scales"].exp()
    gs[3] = gs[3] * torch.sigmoid(params["logit_opacity"]) * torch.sigmoid(-params["logit_opacity"])
    flat = torch.cat([t.reshape(-1) for t in gs]) * c
    m = torch.lerp(flat, d["m"].double(), BETA1)
    v = torch.lerp(flat * flat, d["v"].double(), BETA2)
    upd = m / (1.0 - BETA1 ** STEP) / (torch.sqrt(v / (1.0 - BETA2 ** STEP)) + EPS)
    out, off = {}, 0
    for k in GROUPS:
        n = params[k].numel()
        lr = LR[k] * min(1.0, STEP / WARMUP) if k in ("means", "log_scales") else LR[k]
        out[k] = params[k] - lr * upd[off:off + n].reshape(params[k].shape)
        off += n
    out["quats"] = torch.nn.functional.normalize(out["quats"], dim=1)
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "params": out, "m": m, "v": v,
            "scales": out["log_scales"].exp(), "opacity": torch.sigmoid(out["logit_opacity"])}
