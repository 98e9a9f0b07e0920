"""What is measured of the operators that train a mixer layer, and of the
recurrence that may stand in for its scan.

A mixer layer normalises the residual stream, projects it, runs a recurrence
over the tokens and the gated group-RMSNorm over the recurrence's output.

  recur           h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t for each channel, with
                  a_t = exp(a sigmoid(r_t)); i and r are the logits of the input and decay gates
  recur_step      one token of each sequence, states updated in place
  recur_backward  gradients of x, both gates, a and the states that sequences start from
  ln              layer norm
  ln_backward     gradients of its input, weight and bias
  norm_backward   gradients of the gated group-RMSNorm: both of its modes

Sequences are packed one behind the other (offsets `cu`), their states live in
a pool that `slots` points into, and x, i and r are columns of one projection.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
KEPT = 64  # a training forward pass keeps the state before every 64th row


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _recur(op, rows, width, dtype, seqs=1, tail=0, resume=False):
    return {"op": op, "rows": rows, "width": width, "dtype": dtype, "seqs": seqs, "tail": tail,
            "resume": resume}


def _ln(op, rows, width, dtype):
    return {"op": op, "rows": rows, "width": width, "dtype": dtype}


def _norm(rows, width, group, dtype, mode, packed):
    return {"op": "norm_backward", "rows": rows, "width": width, "group": group, "dtype": dtype,
            "mode": mode, "packed": packed}


def listed():
    def named(name, c):
        return dict(c, name=name)

    return [
        # a prompt of 4096 tokens: one sequence, whose length has to be shared out
        named("recur prompt 4096", _recur("recur", 4096, 7680, "bf16")),
        # ragged prompts packed together, some continuing a cached prefix, rows to spare behind
        named("recur ragged", _recur("recur", 1811, 5120, "f16", seqs=9, tail=13, resume=True)),
        # one decode token, the launch-bound end
        named("recur step 1", _recur("recur_step", 1, 7680, "bf16")),
        # a decode batch
        named("recur step 256", _recur("recur_step", 256, 4800, "f16")),
        # the training step of that prompt
        named("recur backward 4096", _recur("recur_backward", 4096, 7680, "bf16")),
        # odd columns in full precision, as for a check of gradients
        named("recur backward f32 of 1001", _recur("recur_backward", 1025, 1001, "f32", seqs=2,
                                                   resume=True)),
        # the layer's input norm over a training batch
        named("ln 16384", _ln("ln", 16384, 3840, "bf16")),
        # and over one decode token
        named("ln 1", _ln("ln", 1, 3840, "f16")),
        # its gradients over that batch
        named("ln backward 16384", _ln("ln_backward", 16384, 3840, "bf16")),
        # odd columns in full precision
        named("ln backward f32 of 1001", _ln("ln_backward", 333, 1001, "f32")),
        # the gated norm on y and gate as columns of a packed projection, odd groups
        named("norm backward odd span", _norm(16384, 4800, 100, "bf16", "mamba2", True)),
        # the per-head output norm in its ONNX form
        named("norm backward heads of 128", _norm(1023, 4096, 128, "f16", "onnx", False)),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["recur", "recur", "recur_step", "recur_backward", "recur_backward", "ln",
                     "ln_backward", "norm_backward", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    wide = 2 if dtype == "f32" else 1
    if op.startswith("recur"):
        width = rng.choice([512, 1000, 1001, 2560, 3840, 4800, 5120, 7680])
        if op == "recur_step":
            return _recur(op, log_int(1, 256), width, dtype)
        rows = log_int(1, min(16384, 4096 * 7680 // (width * wide)))
        return _recur(op, rows, width, dtype, seqs=min(rng.choice([1, 1, 2, 5, 13]), rows),
                      tail=rng.choice([0, 0, 7]), resume=rng.random() < 0.5)
    if op.startswith("ln"):
        width = rng.choice([100, 960, 1001, 2048, 3840, 4096, 5120, 7680])
        return _ln(op, log_int(1, min(65536, 16384 * 3840 // (width * wide))), width, dtype)
    mode = "mamba2" if dtype == "bf16" else rng.choice(["mamba2", "onnx"])
    width, group = rng.choice([(7680, 960), (5120, 5120), (4096, 128), (4800, 100), (4800, 100),
                               (1001, 77), (7680, 7680), (960, 8)])
    rows = log_int(1, min(65536, 16384 * 4800 // (width * wide)))
    return _norm(rows, width, group, dtype, mode, rng.random() < 0.5)


def _lengths(case):
    """Rows of each sequence: one; equal ones where they divide the rows and
    nothing else is asked; else ragged, with an empty one among five or more."""
    n, rows = case["seqs"], case["rows"]
    if n == 1:
        return [rows]
    if rows % n == 0 and not case["tail"] and not case["resume"]:
        return [rows // n] * n
    r = random.Random(rows * 131 + n)
    parts = n - 1 if n >= 5 else n
    cuts = sorted(r.sample(range(1, rows), parts - 1)) if parts <= rows else list(range(1, rows))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    while len(lens) < n:
        lens.insert(r.randrange(len(lens)), 0)
    return lens


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    T = TYPES[case["dtype"]]
    rows, width = case["rows"], case["width"]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    s = {"case": dict(case)}
    if case["op"].startswith("ln"):
        # a residual stream: channels of different sizes and means
        scale = torch.exp(0.5 * normal(width))
        s["x"] = ((normal(rows, width) + 0.5 * normal(width)) * scale).to(T)
        s["w"], s["b"] = 1 + 0.1 * normal(width), 0.1 * normal(width)
        s["eps"] = 1e-5
        if case["op"] == "ln":
            s["out"] = torch.empty(rows, width, dtype=T, device=DEV)
        else:
            s["dout"] = normal(rows, width).to(T)
        return s
    if case["op"] == "norm_backward":
        inproj = normal(rows, 2 * width + 64).to(T)
        s["inproj"] = inproj
        s["y"], s["gate"] = inproj[:, :width], inproj[:, width:2 * width]
        if not case["packed"]:
            s["y"], s["gate"] = s["y"].contiguous(), s["gate"].contiguous()
        if case["mode"] == "mamba2":
            s["w"], s["eps"] = 1 + 0.1 * normal(width), 1e-5
        else:
            s["w"], s["eps"] = (1 + 0.05 * normal(case["group"])).to(T), 1e-6
        s["dout"] = normal(rows, width).to(T)
        return s

    step = case["op"] == "recur_step"
    lens = [1] * rows if step else _lengths(case)
    nseq, total = len(lens), rows + case["tail"]
    proj = normal(total, 3 * width)
    s["proj"] = proj.to(T)
    s["x"], s["i"], s["r"] = (s["proj"][:, k * width:(k + 1) * width] for k in range(3))
    # decays between 0.9 and 0.999 a token where the gate is open
    u = 0.9 + 0.099 * torch.rand(width, device=DEV, generator=g)
    s["a"] = torch.log(u)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu"] = None if step else torch.tensor(cu, dtype=torch.int32, device=DEV)
    pool = nseq + 2
    s["slots"] = torch.randperm(pool, device=DEV, generator=g)[:nseq].to(torch.int32)
    s["state"] = normal(pool, width)
    s["resume"] = torch.arange(nseq, device=DEV) % 2 == 0 if case["resume"] else None
    if case["op"] != "recur_backward":
        s["out"] = torch.zeros(total, width, dtype=T, device=DEV)
        return s
    s["dout"] = normal(total, width).to(T)
    s["dstate"] = normal(nseq, width)
    # what the forward pass kept: the states before rows 0, 64, 128, ...
    h = torch.cat([torch.zeros(1, width, device=DEV), _states(s)[0]])
    s["saved"] = h[torch.arange(0, total, KEPT, device=DEV).clamp(max=rows)]
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"recur": _recur_plain, "recur_step": _recur_step, "ln": _ln_plain,
                "recur_backward": _recur_backward, "ln_backward": _ln_backward,
                "norm_backward": _norm_backward}[op](s)
    import gated_group_rmsnorm_gb300 as ggrn
    if op == "recur":
        ggrn.linear_recurrence(s["x"], s["i"], s["r"], s["a"], cu_seqlens=s["cu"],
                               state=s["state"], slots=s["slots"], resume=s["resume"],
                               out=s["out"])
        return {"out": s["out"], "state": s["state"]}
    if op == "recur_step":
        ggrn.linear_recurrence_step(s["x"], s["i"], s["r"], s["a"], s["state"], slots=s["slots"],
                                    out=s["out"])
        return {"out": s["out"], "state": s["state"]}
    if op == "recur_backward":
        dx, di, dr, da, dh = ggrn.linear_recurrence_backward(
            s["dout"], s["x"], s["i"], s["r"], s["a"], cu_seqlens=s["cu"], state=s["state"],
            slots=s["slots"], resume=s["resume"], dstate=s["dstate"], saved=s["saved"])
        return {"dx": dx, "di": di, "dr": dr, "da": da, "dh": dh}
    if op == "ln":
        return {"out": ggrn.layer_norm(s["x"], s["w"], s["b"], eps=s["eps"], out=s["out"])}
    if op == "ln_backward":
        dx, dw, db = ggrn.layer_norm_backward(s["dout"], s["x"], s["w"], eps=s["eps"])
        return {"dx": dx, "dw": dw, "db": db}
    dy, dgate, dw = ggrn.backward(s["dout"], s["y"], s["gate"], s["w"],
                                  group_size=s["case"]["group"], eps=s["eps"],
                                  mode=s["case"]["mode"])
    return {"dy": dy, "dgate": dgate, "dw": dw}


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _gates(s):
    """(input gate, decay gate, log decay, decay, sqrt(1 - decay^2)) in 32 bits.  Slow
    decays are next to 1, and a bias of exp's there adds up over a thousand rows:
    1 + expm1 has none."""
    i, r = _sigmoid(s["i"].float()), _sigmoid(s["r"].float())
    p = s["a"] * r
    return i, r, p, 1 + torch.expm1(p), torch.sqrt(-torch.expm1(2 * p))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t down the rows, by doubling."""
    a, h, d = a.clone(), b.clone(), 1
    while d < h.shape[0]:
        h[d:] = h[d:] + a[d:] * h[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return h


def _places(s):
    """First rows of the sequences that have any, whose they are, and their
    starting states; of every sequence its starting state."""
    cu, slots = s["cu"].long(), s["slots"].long()
    h0 = s["state"][slots]
    if s["resume"] is None:
        h0 = torch.zeros_like(h0)
    else:
        h0 = torch.where(s["resume"][:, None], h0, torch.zeros_like(h0))
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(s["case"]["rows"], device=cu.device),
                             right=True)  # of each row
    place = torch.arange(s["case"]["rows"], device=cu.device) - cu[seq]
    return cu, h0, seq, place


def _states(s):
    """h of every row of a sequence, and the sequences' last states."""
    n = s["case"]["rows"]
    i, _, _, a, m = (t[:n] for t in _gates(s))
    cu, h0, seq, place = _places(s)
    first = (place == 0)[:, None]
    b = m * i * s["x"][:n].float()
    h = _scan(torch.where(first, torch.zeros_like(a), a),
              torch.where(first, b + a * h0[seq], b))
    empty = (cu[1:] == cu[:-1])[:, None]
    last = torch.where(empty, h0, h[torch.clamp(cu[1:] - 1, min=0)])
    return h, last


def _recur_plain(s):
    h, last = _states(s)
    s["out"][:h.shape[0]] = h.to(s["out"].dtype)
    s["state"][s["slots"].long()] = last
    return {"out": s["out"], "state": s["state"]}


def _recur_step(s):
    i, _, _, a, m = _gates(s)
    slots = s["slots"].long()
    h = a * s["state"][slots] + m * i * s["x"].float()
    s["state"][slots] = h
    s["out"].copy_(h)
    return {"out": s["out"], "state": s["state"]}


def _recur_backward(s):
    n, T = s["case"]["rows"], s["x"].dtype
    i, r, p, a, m = (t[:n] for t in _gates(s))
    x = s["x"][:n].float()
    cu, h0, seq, place = _places(s)
    first = (place == 0)[:, None]
    last = (torch.arange(n, device=cu.device) == cu[1:][seq] - 1)[:, None]
    h, _ = _states(s)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before = torch.where(first, h0[seq], before)
    # gradients of h: g_t = dout_t + a_{t+1} g_{t+1}, the last one with its state's
    later = torch.cat([a[1:], torch.zeros_like(a[:1])])
    later = torch.where(last, torch.zeros_like(later), later)
    g = s["dout"][:n].float()
    g = torch.where(last, g + s["dstate"][seq], g)
    g = _scan(later.flip(0), g.flip(0)).flip(0)
    dx, di = g * m * i, g * m * x * i * (1 - i)
    # through the decay's logarithm p = a r: a^2 / m grows as m vanishes, p / m does not
    over = torch.where(m > 0, p / m, torch.zeros_like(m))
    dp = g * (before * a * p - i * x * a * a * over)  # the gradient of p, times p
    da = dp.double().sum(0) / s["a"].double()
    dr = dp * (1 - r)
    start = torch.zeros_like(h0)
    start[seq[first[:, 0]]] = (a * g)[first[:, 0]]
    empty = (cu[1:] == cu[:-1])[:, None]
    start = torch.where(empty, s["dstate"], start)
    if s["resume"] is None:
        start = torch.zeros_like(start)
    else:
        start = torch.where(s["resume"][:, None], start, torch.zeros_like(start))
    # (rows of no sequence have gradients of zero)
    spare = torch.zeros(s["case"]["tail"], x.shape[1], device=x.device)
    dx, di, dr = (torch.cat([t, spare]).to(T) for t in (dx, di, dr))
    return {"dx": dx, "di": di, "dr": dr, "da": da.float(), "dh": start}


def _ln_plain(s):
    x = s["x"].float()
    x = x - x.mean(1, keepdim=True)
    v = (x * x).mean(1, keepdim=True)
    s["out"].copy_(x / torch.sqrt(v + s["eps"]) * s["w"] + s["b"])
    return {"out": s["out"]}


def _ln_backward(s):
    x, g = s["x"].float(), s["dout"].float()
    x = x - x.mean(1, keepdim=True)
    inv = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + s["eps"])
    x = x * inv
    u = g * s["w"]
    dx = inv * (u - u.mean(1, keepdim=True) - x * (u * x).mean(1, keepdim=True))
    dw, db = (g * x).sum(0, dtype=torch.float64), g.sum(0, dtype=torch.float64)
    return {"dx": dx.to(s["x"].dtype), "dw": dw.float(), "db": db.float()}


def _norm_backward(s):
    case, T = s["case"], s["y"].dtype
    rows, width, c = case["rows"], case["width"], case["group"]
    y, z, g = s["y"].float(), s["gate"].float(), s["dout"].float()
    sig = _sigmoid(z)
    act, slope = z * sig, sig * (1 + z * (1 - sig))

    def groups(t):
        return t.reshape(rows, width // c, c)

    if case["mode"] == "mamba2":
        v = y * act
        inv = 1 / torch.sqrt((groups(v) ** 2).mean(2, keepdim=True) + s["eps"])
        u = groups(g * s["w"])
        vh = groups(v) * inv
        dv = (inv * (u - vh * (u * vh).mean(2, keepdim=True))).reshape(rows, width)
        dy, dgate = dv * act, dv * y * slope
        dw = (g * vh.reshape(rows, width)).sum(0, dtype=torch.float64)
    else:
        yh = groups(y)
        inv = 1 / torch.sqrt((yh ** 2).mean(2, keepdim=True) + s["eps"])
        yh = yh * inv
        w = s["w"].float()
        u = groups(g * act) * w
        dy = (inv * (u - yh * (u * yh).mean(2, keepdim=True))).reshape(rows, width)
        dgate = (yh * w).reshape(rows, width) * g * slope
        dw = (groups(g * act) * yh).sum((0, 1), dtype=torch.float64)
    return {"dy": dy.to(T), "dgate": dgate.to(T), "dw": dw.float()}


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits: tokens one after the other, and
# gradients by differentiating the definition.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if not op.startswith("recur"):
        return _exact_norm(s, op)
    n, step, back = case["rows"], op == "recur_step", op == "recur_backward"
    x, zi, zr = (s[k][:n].double().requires_grad_(back) for k in ("x", "i", "r"))
    rate = s["a"].double().requires_grad_(back)
    slots = s["slots"].long()
    with torch.set_grad_enabled(back):
        log = rate * torch.sigmoid(zr)
        a, b = torch.exp(log), torch.sqrt(-torch.expm1(2 * log)) * torch.sigmoid(zi) * x
        lens = [1] * n if step else _lengths(case)
        start = s["state"][slots].double()
        if not step:
            keep = s["resume"] if s["resume"] is not None else torch.zeros_like(slots,
                                                                                dtype=torch.bool)
            start = start * keep[:, None]
        start.requires_grad_(back)
        if step:
            h = a * start + b
            last = h
        else:
            at, bt, rows, last = a.unbind(0), b.unbind(0), [], []
            t = 0
            for h0, length in zip(start.unbind(0), lens):
                for _ in range(length):
                    h0 = at[t] * h0 + bt[t]
                    rows.append(h0)
                    t += 1
                last.append(h0)
            h, last = torch.stack(rows), torch.stack(last)
        if not back:
            out, state = s["out"].double(), s["state"].double()
            out[:n], state[slots] = h, last
            return {"out": out, "state": state}
        dx, di, dr, da, dh = torch.autograd.grad(
            [h, last], [x, zi, zr, rate, start], [s["dout"][:n].double(), s["dstate"].double()])
    dx, di, dr = (torch.nn.functional.pad(t, (0, 0, 0, case["tail"])) for t in (dx, di, dr))
    return {"dx": dx, "di": di, "dr": dr, "da": da, "dh": dh * keep[:, None]}


def _exact_norm(s, op):
    case = s["case"]
    back = op != "ln"
    with torch.set_grad_enabled(back):
        w = s["w"].double().requires_grad_(back)
        if op.startswith("ln"):
            x, b = s["x"].double().requires_grad_(back), s["b"].double().requires_grad_(back)
            var, mean = torch.var_mean(x, dim=1, keepdim=True, correction=0)
            out = (x - mean) * torch.rsqrt(var + s["eps"]) * w + b
            if not back:
                return {"out": out}
            dx, dw, db = torch.autograd.grad(out, [x, w, b], s["dout"].double())
            return {"dx": dx, "dw": dw, "db": db}
        y, z = s["y"].double().requires_grad_(True), s["gate"].double().requires_grad_(True)
        act = z * torch.sigmoid(z)
        v = (y * act if case["mode"] == "mamba2" else y).unflatten(1, (-1, case["group"]))
        v = v * torch.rsqrt((v * v).mean(2, keepdim=True) + s["eps"])
        out = v.flatten(1) * w if case["mode"] == "mamba2" else (v * w).flatten(1) * act
        dy, dgate, dw = torch.autograd.grad(out, [y, z, w], s["dout"].double())
        return {"dy": dy, "dgate": dgate, "dw": dw}


def work(case):
    """Bytes: inputs and outputs once, a state once in (where it is read) and
    once out.  Operations: about what one element's formulas hold."""
    es = BYTES[case["dtype"]]
    rows, width, op = case["rows"], case["width"], case["op"]
    n = rows * width
    if op == "ln":
        return {"bytes": 2 * n * es + 8 * width, "flops": 8 * n}
    if op == "ln_backward":
        return {"bytes": 3 * n * es + 12 * width, "flops": 16 * n}
    if op == "norm_backward":
        w = width * 4 if case["mode"] == "mamba2" else case["group"] * es
        dw = width * 4 if case["mode"] == "mamba2" else case["group"] * 4
        return {"bytes": 5 * n * es + w + dw, "flops": 25 * n}
    nseq = rows if op == "recur_step" else case["seqs"]
    read = nseq if op == "recur_step" else (nseq + 1) // 2 if case["resume"] else 0
    if op == "recur_backward":
        kept = (rows + KEPT - 1) // KEPT
        return {"bytes": 7 * n * es + 4 * width * (2 + kept + read + 2 * nseq), "flops": 45 * n}
    return {"bytes": 4 * n * es + 4 * width * (1 + read + nseq), "flops": 20 * n}
