"""What is measured of the Mamba-2 mixer's operators around the gated norm.

The mixer packs one in-proj row per token as [z | x B C | dt].  Before the
gated group-RMSNorm it runs a short causal convolution with SiLU over the
x B C columns and the selective state space scan over its output:

  conv       prompts: out[t, c] = silu(bias[c] + sum_k w[c, k] x[t - (W-1) + k, c])
  conv_step  one token a sequence, from the last W-1 inputs of each
  scan       prompts: S_t = exp(dt_t a) S_{t-1} + dt_t x_t B_t^T, y_t = S_t C_t + D x_t
  scan_step  one token a sequence, the state updated in place

Sequences are packed one behind the other (offsets `cu`), and their states
live in a pool that `slots` points into.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
CHUNK = 64  # rows of a chunk of the plain scan


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _case(op, rows, heads, head_dim, groups, state, dtype, seqs=1, tail=0, resume=False, taps=4):
    return {"op": op, "rows": rows, "heads": heads, "head_dim": head_dim, "groups": groups,
            "state": state, "dtype": dtype, "seqs": seqs, "tail": tail, "resume": resume,
            "taps": taps}


def listed():
    def named(name, c):
        return dict(c, name=name)

    return [
        # a prompt of 4096 tokens through the mixer whose norm has 7680 columns in 8 groups
        named("conv prompt 4096", _case("conv", 4096, 96, 80, 8, 128, "bf16")),
        # ragged prompts packed together, some continuing a cached prefix, rows to spare behind
        named("conv ragged", _case("conv", 1811, 80, 64, 1, 128, "f16", seqs=9, tail=13,
                                   resume=True)),
        # one decode token, the launch-bound end
        named("conv step 1", _case("conv_step", 1, 96, 80, 8, 128, "bf16")),
        # a decode batch
        named("conv step 256", _case("conv_step", 256, 96, 80, 8, 128, "bf16")),
        # the scan of the 4096-token prompt: one sequence, so its length has to be split
        named("scan prompt 4096", _case("scan", 4096, 96, 80, 8, 128, "bf16")),
        # eight prompts of 2048 tokens: the largest amount of work
        named("scan batch 8x2048", _case("scan", 16384, 80, 64, 1, 128, "bf16", seqs=8)),
        # ragged prompts, some continuing a cached prefix, one of them empty
        named("scan ragged", _case("scan", 3777, 96, 80, 8, 128, "bf16", seqs=11, tail=9,
                                   resume=True)),
        # a prompt shorter than any tile
        named("scan prompt 37", _case("scan", 37, 80, 64, 1, 128, "bf16")),
        # f32 (a check in full precision) with the odd span of 100 as head size
        named("scan f32 heads of 100", _case("scan", 1025, 48, 100, 1, 64, "f32", seqs=2)),
        # one decode token
        named("scan step 1", _case("scan_step", 1, 96, 80, 8, 128, "bf16")),
        # a decode batch: the state's bytes
        named("scan step 128", _case("scan_step", 128, 96, 80, 8, 128, "bf16")),
        # a small f16 batch with 128-wide heads
        named("scan step 7 f16", _case("scan_step", 7, 32, 128, 1, 64, "f16")),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step"])
    head_dim = rng.choice([64, 64, 80, 96, 100, 128])
    groups = rng.choice([1, 2, 4, 8])
    heads = groups * rng.randint(max(1, 16 // groups), 96 // groups)
    state = rng.choice([16, 64, 96, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    taps = rng.choice([2, 3, 4, 4])
    width = heads * head_dim
    if op in ("conv_step", "scan_step"):
        # what a batch of the largest listed step holds in states
        most = 256 if op == "conv_step" else max(1, min(256, 128 * 96 * 80 * 128 // (width * state)))
        return _case(op, log_int(1, most), heads, head_dim, groups, state, dtype, taps=taps)
    most = 16384 * 5120 // width
    if op == "scan" and dtype != "bf16":
        most //= 4
    rows = log_int(1, min(most, 16384))
    seqs = min(rng.choice([1, 1, 2, 5, 13]), rows)
    return _case(op, rows, heads, head_dim, groups, state, dtype, seqs=seqs,
                 tail=rng.choice([0, 0, 7]), resume=rng.random() < 0.5, taps=taps)


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


def _dims(case):
    inner = case["heads"] * case["head_dim"]
    gn = case["groups"] * case["state"]
    return inner, gn, inner + 2 * gn


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    T = TYPES[case["dtype"]]
    inner, gn, cd = _dims(case)
    heads, rows, taps = case["heads"], case["rows"], case["taps"]
    step = case["op"].endswith("_step")
    total = rows + case["tail"]

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    s = {"case": dict(case)}
    # the packed in-proj output [z | x B C | dt]
    s["inproj"] = normal(total, inner + cd + heads).to(T)
    # where sequences lie and which slots of the pool are theirs
    if step:
        nseq = rows
        s["cu"] = None
    else:
        lens = _lengths(case)
        nseq = len(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    pool = nseq + 2
    s["slots"] = torch.randperm(pool, device=DEV, generator=g)[:nseq].to(torch.int32)
    s["resume"] = None
    if case["resume"]:
        s["resume"] = torch.arange(nseq, device=DEV) % 2 == 0
    if case["op"].startswith("conv"):
        s["x"] = s["inproj"][:, inner:inner + cd]
        s["weight"] = normal(cd, taps) / math.sqrt(taps)
        s["bias"] = 0.1 * normal(cd)
        s["state"] = normal(pool, taps - 1, cd).to(T)
        s["out"] = torch.zeros(total, cd, dtype=T, device=DEV)
        return s
    # the scan reads the convolution's output (after its SiLU) and the raw dt columns
    s["xbc"] = torch.nn.functional.silu(normal(total, cd)).to(T)
    s["x"], s["b"], s["c"] = s["xbc"][:, :inner], s["xbc"][:, inner:inner + gn], s["xbc"][:, inner + gn:]
    s["dt"] = s["inproj"][:, inner + cd:]
    u = torch.rand(heads, device=DEV, generator=g)
    dt0 = torch.exp(u * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    s["a"] = -(1 + 15 * torch.rand(heads, device=DEV, generator=g))
    s["d"] = 1 + 0.1 * normal(heads)
    s["state"] = 0.3 * normal(pool, heads, case["head_dim"], case["state"])
    s["out"] = torch.zeros(total, inner, dtype=T, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    op, case = s["case"]["op"], s["case"]
    if own:
        import gated_group_rmsnorm_gb300 as ggrn
        if op == "conv":
            ggrn.causal_conv(s["x"], s["weight"], s["bias"], activation="silu", cu_seqlens=s["cu"],
                             state=s["state"], slots=s["slots"], resume=s["resume"], out=s["out"])
        elif op == "conv_step":
            ggrn.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], activation="silu",
                                  slots=s["slots"], out=s["out"])
        elif op == "scan":
            ggrn.ssm_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], head_dim=case["head_dim"],
                          state_size=case["state"], d=s["d"], dt_bias=s["dt_bias"],
                          cu_seqlens=s["cu"], state=s["state"], slots=s["slots"],
                          resume=s["resume"], out=s["out"])
        else:
            ggrn.ssm_scan_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], d=s["d"],
                               dt_bias=s["dt_bias"], slots=s["slots"], out=s["out"])
    else:
        {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step}[op](s)
    return {"out": s["out"], "state": s["state"]}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _sequence_of_rows(cu, rows):
    """(sequence, place in it, whether it has one) of each packed row."""
    r = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), r.to(cu.dtype), right=True)
    fine = seq < cu.numel() - 1
    seq = torch.clamp(seq, max=cu.numel() - 2)
    return seq, r - cu[seq].long(), fine


def _conv(s):
    x, cu, taps = s["x"].float(), s["cu"].long(), s["weight"].shape[1]
    rows, cd = x.shape
    slots = s["slots"].long()
    seq, pos, fine = _sequence_of_rows(s["cu"], rows)
    # one table of rows: the inputs, each sequence's old state, a row of zeros
    old = s["state"].float()[slots]
    if s["resume"] is None:
        old = torch.zeros_like(old)
    else:
        old = torch.where(s["resume"][:, None, None], old, torch.zeros_like(old))
    table = torch.cat([x, old.reshape(-1, cd)])

    def window(q, p, n):  # table rows of the n inputs that end just before place p of sequence q
        t = p[:, None] - n + torch.arange(n, device=p.device)
        return torch.where(t >= 0, cu[q][:, None] + t, rows + q[:, None] * (taps - 1) + taps - 1 + t)

    got = table[window(seq, pos + 1, taps)]                      # [rows, taps, cd]
    v = _silu((got * s["weight"].t()).sum(1) + s["bias"]).to(s["out"].dtype)
    q = torch.arange(cu.numel() - 1, device=x.device)
    new = table[window(q, cu[1:] - cu[:-1], taps - 1)].to(s["state"].dtype)
    s["out"].copy_(torch.where(fine[:, None], v, s["out"]))
    s["state"][slots] = new


def _conv_step(s):
    slots = s["slots"].long()
    got = torch.cat([s["state"][slots].float(), s["x"].float()[:, None]], 1)
    s["out"].copy_(_silu((got * s["weight"].t()).sum(1) + s["bias"]))
    s["state"][slots] = got[:, 1:].to(s["state"].dtype)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _scan(s):
    """In chunks of CHUNK rows of one sequence: within a chunk as a masked
    product, between chunks through their states, both in 32 bits with the
    decays' exponents in 64."""
    case, Q = s["case"], CHUNK
    H, P, G, N = case["heads"], case["head_dim"], case["groups"], case["state"]
    cu, slots = s["cu"].long(), s["slots"].long()
    dev, rows, nseq = cu.device, s["x"].shape[0], cu.numel() - 1
    nc = rows // Q + nseq                                        # as many chunks at most
    per = (cu[1:] - cu[:-1] + Q - 1) // Q                        # chunks of each sequence
    ends = torch.cumsum(per, 0)
    k = torch.arange(nc, device=dev)
    seq = torch.searchsorted(ends, k, right=True)
    used = seq < nseq
    seq = torch.clamp(seq, max=nseq - 1)
    at = cu[seq] + (k - (ends - per)[seq]) * Q
    row = at[:, None] + torch.arange(Q, device=dev)              # [nc, Q]
    fine = (row < cu[1:][seq][:, None]) & used[:, None]
    row = torch.where(fine, row, torch.zeros_like(row))

    def rows_of(t, *shape):
        v = t[row].float().reshape(nc, Q, *shape)
        return torch.where(fine.reshape(nc, Q, *[1] * len(shape)), v, torch.zeros_like(v))

    x, b, c = rows_of(s["x"], H, P), rows_of(s["b"], G, N), rows_of(s["c"], G, N)
    dt = _softplus(s["dt"][row].double() + s["dt_bias"].double())
    dt = torch.where(fine[:, :, None], dt, torch.zeros_like(dt))  # [nc, Q, H]
    cs = torch.cumsum(dt * s["a"].double(), 1).transpose(1, 2)   # [nc, H, Q]
    xh = x.transpose(1, 2)                                       # [nc, H, Q, P]
    dth = dt.transpose(1, 2)
    lower = torch.tril(torch.ones(Q, Q, dtype=torch.bool, device=dev))
    gap = torch.where(lower, cs[..., :, None] - cs[..., None, :], cs.new_tensor(-math.inf))
    m = (torch.exp(gap) * dth[..., None, :]).float()             # [nc, H, Q, Q]
    cb = torch.matmul(c.transpose(1, 2), b.permute(0, 2, 3, 1))  # [nc, G, Q, Q]
    m = (m.reshape(nc, G, H // G, Q, Q) * cb[:, :, None]).reshape(nc, H, Q, Q)
    y = torch.matmul(m, xh)
    # what each chunk adds to the state by its end
    w = (torch.exp(cs[..., -1:] - cs) * dth).float()
    bh = b.transpose(1, 2).repeat_interleave(H // G, 1)          # [nc, H, Q, N]
    add = torch.matmul((xh * w[..., None]).transpose(2, 3), bh)  # [nc, H, P, N]
    # the states at chunk starts and sequence ends, from the old states and the sums
    old = s["state"][slots]
    if s["resume"] is None:
        old = torch.zeros_like(old)
    else:
        old = torch.where(s["resume"][:, None, None, None], old, torch.zeros_like(old))
    total = torch.where(used[:, None], cs[..., -1], torch.zeros_like(cs[..., -1]))  # [nc, H]
    sums = torch.cat([torch.zeros_like(total[:1]), torch.cumsum(total, 0)])  # before each chunk
    src_after = torch.cat([sums[1:], sums[(ends - per)]])        # decay counted from here
    src_seq = torch.cat([seq, torch.arange(nseq, device=dev)])
    src_at = torch.cat([k, torch.full((nseq,), -1, device=dev)])
    src_ok = torch.cat([used, torch.ones(nseq, dtype=torch.bool, device=dev)])
    dst_at = torch.cat([k, torch.full((nseq,), nc, device=dev)])
    dst_seq = src_seq
    dst_sum = torch.cat([sums[:-1], sums[ends]])
    ok = (dst_seq[:, None] == src_seq) & (src_at < dst_at[:, None]) & src_ok
    gap = torch.where(ok[..., None], dst_sum[:, None] - src_after[None], sums.new_tensor(-math.inf))
    carry = torch.exp(gap).float().permute(2, 0, 1)              # [H, dst, src]
    src = torch.cat([add, old]).transpose(0, 1).reshape(H, nc + nseq, P * N)
    got = torch.matmul(carry, src).reshape(H, nc + nseq, P, N).transpose(0, 1)
    start, final = got[:nc], got[nc:]
    # their share of the rows' outputs
    ch = c.transpose(1, 2).repeat_interleave(H // G, 1)
    y = y + torch.exp(cs).float()[..., None] * torch.matmul(ch, start.transpose(2, 3))
    y = y + s["d"][:, None, None] * xh
    y = y.transpose(1, 2).reshape(nc, Q, H * P).to(s["out"].dtype)
    s["out"][row[fine]] = y[fine]
    s["state"][slots] = final


def _scan_step(s):
    case = s["case"]
    H, P, G, N = case["heads"], case["head_dim"], case["groups"], case["state"]
    n, slots = s["x"].shape[0], s["slots"].long()
    x = s["x"].float().reshape(n, H, P)
    b = s["b"].float().reshape(n, G, 1, N).expand(n, G, H // G, N).reshape(n, H, N)
    c = s["c"].float().reshape(n, G, 1, N).expand(n, G, H // G, N).reshape(n, H, N)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    new = s["state"][slots] * torch.exp(dt * s["a"])[..., None, None]
    new = new + (dt[..., None] * x)[..., None] * b[:, :, None]
    s["state"][slots] = new
    y = (new * c[:, :, None]).sum(-1) + s["d"][:, None] * x
    s["out"].copy_(y.reshape(n, H * P))


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits, one token after the other.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    out, state = s["out"].double(), s["state"].double()
    step = case["op"].endswith("_step")
    if step:
        lens, starts = [1] * case["rows"], list(range(case["rows"]))
    else:
        lens = _lengths(case)
        starts = [sum(lens[:i]) for i in range(len(lens))]
    slots = s["slots"].long()
    live = state[slots]
    if not step:
        keep = s["resume"] if s["resume"] is not None else torch.zeros_like(slots, dtype=torch.bool)
        live = torch.where(keep.reshape(-1, *[1] * (live.dim() - 1)), live, torch.zeros_like(live))
    # longest first, so that the sequences still running are a prefix
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    live = live[torch.tensor(order, device=DEV)]
    first = torch.tensor([starts[i] for i in order], device=DEV)
    H, P, G, N = case["heads"], case["head_dim"], case["groups"], case["state"]
    for t in range(max(lens)):
        n = sum(ln > t for ln in lens)
        rows = first[:n] + t
        x = s["x"][rows].double()
        if case["op"].startswith("conv"):
            hist = torch.cat([live[:n], x[:, None]], 1)
            v = torch.einsum("nkc,ck->nc", hist, s["weight"].double()) + s["bias"].double()
            out[rows] = v * torch.sigmoid(v)
            live[:n] = hist[:, 1:]
            continue
        x = x.reshape(n, H, P)
        grp = torch.arange(H, device=DEV) // (H // G)
        b = s["b"][rows].double().reshape(n, G, N)[:, grp]
        c = s["c"][rows].double().reshape(n, G, N)[:, grp]
        v = s["dt"][rows].double() + s["dt_bias"].double()
        dt = torch.logaddexp(v, torch.zeros_like(v))
        cur = live[:n]
        cur.mul_(torch.exp(dt * s["a"].double())[..., None, None])
        cur.addcmul_((dt[..., None] * x)[..., None], b[:, :, None, :])
        y = torch.matmul(cur, c[..., None])[..., 0] + s["d"].double()[:, None] * x
        out[rows] = y.reshape(n, H * P)
    state[slots[torch.tensor(order, device=DEV)]] = live
    return {"out": out, "state": state}


def work(case):
    """Bytes: inputs and outputs once, a state once in (where it is read) and
    once out.  Operations of the scan: the recurrence's own, a multiplication
    and two fused multiply-adds for each entry of the state."""
    es = BYTES[case["dtype"]]
    inner, gn, cd = _dims(case)
    rows, heads, taps = case["rows"], case["heads"], case["taps"]
    step = case["op"].endswith("_step")
    nseq = rows if step else case["seqs"]
    read = nseq if step else (nseq + 1) // 2 if case["resume"] else 0
    if case["op"].startswith("conv"):
        held = (taps - 1) * cd * es
        return {"bytes": 2 * rows * cd * es + cd * (taps + 1) * 4 + (nseq + read) * held,
                "flops": rows * cd * (2 * taps + 4)}
    held = inner * case["state"] * 4
    return {"bytes": rows * (2 * inner + 2 * gn + heads) * es + 12 * heads + (nseq + read) * held,
            "flops": rows * inner * (5 * case["state"] + 2)}
