"""The layer operators around the KDA recurrence, measured: the short causal convolution, the
selective state space scan (both for prompts and for single tokens, over slot-indexed state
pools) and the root-mean-square norm with residual, gate and 8-bit output.

``run`` calls the framework's operators where ``own`` is true and computes their plain form with
elementary torch operations where it is false.  ``exact`` computes the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -40


def _lens(c):
    """The sequence lengths of a prompt case (part of the case, not of its seed)."""
    r = random.Random(c["len_seed"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"] - 1)] + [c["hi"]]


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the q, k and v rows of 12 heads of 128, of 16 ragged prompts of which some continue
        # from their pool slot: the convolution before a KDA prefill
        dict(name="conv prompts bf16", op="conv_prefill", dtype="bf16", seqs=16, lo=1, hi=4096,
             len_seed=7, channels=4608, width=4, parts=3, pool=24, silu=True, bias=False),
        # one short prompt in 32 bits with an odd channel count: latency, unaligned rows
        dict(name="conv one short f32", op="conv_prefill", dtype="f32", seqs=1, lo=77, hi=77,
             len_seed=1, channels=1003, width=3, parts=1, pool=1, silu=False, bias=True),
        # a decode step of a large batch, one token each
        dict(name="conv step bf16", op="conv_decode", dtype="bf16", seqs=1024, tokens=1,
             channels=4608, width=4, parts=3, pool=1100, silu=True, bias=False),
        # verification of three drafts of a few requests
        dict(name="conv drafts f16", op="conv_decode", dtype="f16", seqs=9, tokens=4,
             channels=2048, width=4, parts=1, pool=12, silu=True, bias=True),
        # one long prompt through a wide scan
        dict(name="scan one long bf16", op="scan_prefill", dtype="bf16", seqs=1, lo=8192, hi=8192,
             len_seed=1, channels=4096, size=16, groups=1, pool=1, gate=True),
        # ragged prompts in one packed batch
        dict(name="scan prompts f16", op="scan_prefill", dtype="f16", seqs=16, lo=1, hi=4096,
             len_seed=7, channels=2048, size=16, groups=1, pool=20, gate=True),
        # a small scan in 32 bits, odd sizes, no gate
        dict(name="scan short odd f32", op="scan_prefill", dtype="f32", seqs=2, lo=30, hi=90,
             len_seed=3, channels=250, size=13, groups=2, pool=3, gate=False),
        # a decode step of a large batch
        dict(name="scan step bf16", op="scan_decode", dtype="bf16", seqs=256, tokens=1,
             channels=4096, size=16, groups=1, pool=300, gate=True),
        # verification of three drafts of a few requests, a wider state
        dict(name="scan drafts bf16", op="scan_decode", dtype="bf16", seqs=8, tokens=4,
             channels=1536, size=64, groups=4, pool=8, gate=True),
        # the norm before the projections of a layer, with the residual stream's addition
        dict(name="norm residual bf16", op="rms_norm", dtype="bf16", tokens=8192, heads=1,
             width=4096, residual=True, gate="none", bits8=False, group=0),
        # the gated norm of the heads of a KDA prefill of 8 x 4096 tokens, in 8 bits for the
        # output projection
        dict(name="norm heads gated e4m3", op="rms_norm", dtype="bf16", tokens=32768, heads=12,
             width=128, residual=False, gate="sigmoid", bits8=True, group=128),
        # a decode step's rows in 8 bits with one scale a row, odd width
        dict(name="norm rows e4m3 f16", op="rms_norm", dtype="f16", tokens=33, heads=1,
             width=2500, residual=True, gate="none", bits8=True, group=0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prefill", "conv_decode", "scan_prefill", "scan_decode", "rms_norm"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    c = dict(op=op, dtype=dt)
    if op == "conv_prefill":
        ch, parts = _logint(rng, 64, 8192), rng.choice([1, 1, 3])
        ch = max(parts, ch - ch % (parts * rng.choice([1, 8])))
        seqs = _logint(rng, 1, 64)
        hi = _logint(rng, 1, max(2, min(8192, 50_000_000 // (ch * seqs))))
        c.update(seqs=seqs, lo=rng.choice([0, 1, hi]), hi=hi, len_seed=rng.randrange(1 << 20),
                 channels=ch, width=rng.choice([2, 3, 4, 4]), parts=parts,
                 pool=seqs + rng.randrange(4), silu=rng.random() < 0.7, bias=rng.random() < 0.5)
    elif op == "conv_decode":
        ch, parts = _logint(rng, 64, 8192), rng.choice([1, 1, 3])
        ch = max(parts, ch - ch % (parts * rng.choice([1, 8])))
        seqs = _logint(rng, 1, 1024)
        c.update(seqs=seqs, tokens=rng.choice([1, 1, 2, 4, 7]), channels=ch,
                 width=rng.choice([2, 3, 4, 4]), parts=parts, pool=seqs + rng.randrange(9),
                 silu=rng.random() < 0.7, bias=rng.random() < 0.5)
    elif op == "scan_prefill":
        groups = rng.choice([1, 1, 2, 4])
        size = rng.choice([16, 16, 16, 8, 5, 32, 64, 128])
        ch = _logint(rng, 16, 4096)
        ch = max(groups, ch - ch % (groups * rng.choice([1, 8])))
        seqs = _logint(rng, 1, 32)
        hi = _logint(rng, 1, max(2, min(8192, 400_000_000 // (ch * seqs * size))))
        c.update(seqs=seqs, lo=rng.choice([0, 1, hi]), hi=hi, len_seed=rng.randrange(1 << 20),
                 channels=ch, size=size, groups=groups, pool=seqs + rng.randrange(4),
                 gate=rng.random() < 0.7)
    elif op == "scan_decode":
        groups = rng.choice([1, 1, 2, 4])
        size = rng.choice([16, 16, 16, 8, 5, 32, 64, 128])
        ch = _logint(rng, 16, 4096)
        ch = max(groups, ch - ch % (groups * rng.choice([1, 8])))
        seqs = _logint(rng, 1, max(2, min(1024, 16_000_000 // (ch * size))))
        c.update(seqs=seqs, tokens=rng.choice([1, 1, 2, 4, 7]), channels=ch, size=size,
                 groups=groups, pool=seqs + rng.randrange(9), gate=rng.random() < 0.7)
    else:
        heads = rng.choice([1, 1, 4, 12])
        width = _logint(rng, 32, 16384) if heads == 1 else rng.choice([64, 128, 128, 200])
        if rng.random() < 0.6:
            width = max(8, width - width % 8)
        bits8 = rng.random() < 0.5
        c.update(tokens=_logint(rng, 1, max(2, 25_000_000 // (heads * width))), heads=heads,
                 width=width, residual=rng.random() < 0.5,
                 gate=rng.choice(["none", "none", "silu", "sigmoid"]), bits8=bits8,
                 group=rng.choice([0, 128]) if bits8 else 0)
    return c


# ---------------------------------------------------------------- inputs
def _conv_params(c, g):
    w = torch.randn(c["channels"], c["width"], generator=g, device="cuda") / math.sqrt(c["width"])
    b = 0.1 * torch.randn(c["channels"], generator=g, device="cuda") if c["bias"] else None
    return w, b


def _scan_params(c, g):
    """Parameters as such models start from: A = -(1 .. size), steps between 1e-3 and 1e-1."""
    D, S = c["channels"], c["size"]
    A_log = torch.log(torch.arange(1, S + 1, device="cuda", dtype=torch.float32)).repeat(D, 1)
    A_log += 0.1 * torch.randn(D, S, generator=g, device="cuda")
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(D, generator=g, device="cuda"))
    dt_bias = dt + torch.log(-torch.expm1(-dt))
    skip = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    return A_log, dt_bias, skip


def _scan_rows(c, rows, g):
    """Activations as slices of the rows that projections write: x beside z, dt on its own,
    B beside C behind the low-rank part of dt."""
    D, S, G, t = c["channels"], c["size"], c["groups"], DTYPES[c["dtype"]]
    xz = torch.randn(rows, 2 * D, generator=g, device="cuda")
    xz[:, :D] = torch.nn.functional.silu(xz[:, :D])
    xz = xz.to(t)
    dt = (0.5 * torch.randn(rows, D, generator=g, device="cuda")).to(t)
    rank = 8 * max(1, D // 128)
    low = torch.randn(rows, rank + 2 * G * S, generator=g, device="cuda").to(t)
    B = low[:, rank:rank + G * S].unflatten(1, (G, S))
    C = low[:, rank + G * S:].unflatten(1, (G, S))
    return xz[:, :D], dt, (xz[:, D:] if c["gate"] else None), B, C


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"].endswith("prefill"):
        lens = _lens(c)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_len=max(lens),
                 slots=torch.randperm(c["pool"], generator=g, device="cuda")[:c["seqs"]].int(),
                 has=torch.rand(c["seqs"], generator=g, device="cuda") < 0.5)
        rows = cu[-1]
    elif c["op"].endswith("decode"):
        s.update(slots=torch.randperm(c["pool"], generator=g, device="cuda")[:c["seqs"]].int())
        if c["seqs"] > 2:
            s["slots"][1] = -1          # a padding row of the batch
        rows = c["seqs"] * c["tokens"]
    if c["op"].startswith("conv"):
        t = DTYPES[c["dtype"]]
        s["x"] = torch.randn(rows, c["channels"], generator=g, device="cuda").to(t)
        s["w"], s["b"] = _conv_params(c, g)
        s["pool"] = torch.randn(c["pool"], c["width"] - 1, c["channels"], generator=g,
                                device="cuda").to(t)
    elif c["op"].startswith("scan"):
        s["x"], s["dt"], s["z"], s["B"], s["C"] = _scan_rows(c, rows, g)
        s["A_log"], s["dt_bias"], s["skip"] = _scan_params(c, g)
        s["pool"] = 0.1 * torch.randn(c["pool"], c["channels"], c["size"], generator=g,
                                      device="cuda")
    else:
        t, shp = DTYPES[c["dtype"]], (c["tokens"], c["heads"], c["width"])
        s["x"] = torch.randn(*shp, generator=g, device="cuda").to(t)
        s["res"] = (3 * torch.randn(*shp, generator=g, device="cuda")).to(t) \
            if c["residual"] else None
        s["gate"] = torch.randn(*shp, generator=g, device="cuda").to(t) \
            if c["gate"] != "none" else None
        s["w"] = 1 + 0.1 * torch.randn(c["width"], generator=g, device="cuda")
    if c["op"].endswith("decode"):
        for k in ("x", "dt", "z", "B", "C"):
            if s.get(k) is not None:
                s[k] = s[k].unflatten(0, (c["seqs"], c["tokens"]))
    return s


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import kda_chunked_recurrent_b200 as K
    c = s["case"]
    op = c["op"]
    if op == "conv_prefill":
        out = K.conv_prefill(s["x"], s["w"], bias=s["b"], state=s["pool"],
                             state_indices=s["slots"], has_state=s["has"], cu_seqlens=s["cu"],
                             parts=c["parts"], silu=c["silu"])
        return out, s["pool"]
    if op == "conv_decode":
        out, _ = K.conv_decode(s["x"], s["w"], s["pool"], bias=s["b"], state_indices=s["slots"],
                               parts=c["parts"], silu=c["silu"])
        return out, s["pool"]
    if op == "scan_prefill":
        out = K.scan_prefill(s["x"], s["dt"], s["A_log"], s["B"], s["C"], D=s["skip"], z=s["z"],
                             dt_bias=s["dt_bias"], state=s["pool"], state_indices=s["slots"],
                             has_state=s["has"], cu_seqlens=s["cu"], max_seqlen=s["max_len"])
        return out, s["pool"]
    if op == "scan_decode":
        out, _ = K.scan_decode(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["pool"],
                               D=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                               state_indices=s["slots"])
        return out, s["pool"]
    out, res, scales = K.rms_norm(s["x"], s["w"], eps=1e-6, residual=s["res"], gate=s["gate"],
                                  gate_activation=c["gate"] if c["gate"] != "none" else "silu",
                                  out_dtype=torch.float8_e4m3fn if c["bits8"] else None,
                                  group=c["group"])
    return [t for t in (out, res, scales) if t is not None]


# ---------------------------------------------------------------- the plain forms
def _split(y, parts):
    """[..., C] as [parts, ..., C / parts]."""
    return y if parts == 1 else y.unflatten(-1, (parts, -1)).movedim(-2, 0).contiguous()


def _window_sum(ext, end, s):
    """sum_j w[c, j] ext[end - (W - 1) + j, c] (+ bias) (SiLU), rounded once."""
    c = s["case"]
    W = c["width"]
    rows = end[:, None] + torch.arange(1 - W, 1, device=ext.device)
    y = (ext[rows] * s["w"].t()).sum(1)
    if s["b"] is not None:
        y = y + s["b"]
    if c["silu"]:
        y = y * torch.sigmoid(y)
    return y.to(s["x"].dtype)


def _plain_conv_prefill(s):
    c = s["case"]
    W, N, x, cu = c["width"], c["seqs"], s["x"].float(), s["cu"].long()
    T, slots = x.shape[0], s["slots"].long()
    old = s["pool"][slots].float() * s["has"][:, None, None]
    # every sequence's state rows, then its inputs
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(T, device=x.device), right=True)
    at = torch.arange(T, device=x.device) + (seq + 1) * (W - 1)
    first = cu[:-1] + torch.arange(N, device=x.device) * (W - 1)
    ext = x.new_empty(T + N * (W - 1), x.shape[1])
    ext[at] = x
    ext[first[:, None] + torch.arange(W - 1, device=x.device)] = old
    out = _split(_window_sum(ext, at, s), c["parts"])
    last = cu[1:] + (torch.arange(N, device=x.device) + 1) * (W - 1)
    s["pool"][slots] = ext[last[:, None] + torch.arange(1 - W, 0, device=x.device)].to(
        s["pool"].dtype)
    return out, s["pool"]


def _plain_conv_decode(s):
    c = s["case"]
    W, N, T = c["width"], c["seqs"], c["tokens"]
    live = s["slots"] >= 0
    slots = s["slots"].long().clamp(min=0)
    ext = torch.cat([s["pool"][slots].float(), s["x"].float()], 1)      # [N, W - 1 + T, C]
    at = (torch.arange(N, device=ext.device)[:, None] * (W - 1 + T) + W - 1
          + torch.arange(T, device=ext.device)).flatten()
    y = _window_sum(ext.flatten(0, 1), at, s).unflatten(0, (N, T))
    y = torch.where(live[:, None, None], y, torch.zeros_like(y))
    s["pool"][slots[live]] = ext[live][:, T:].to(s["pool"].dtype)
    return _split(y, c["parts"]), s["pool"]


def _steps(s):
    """Decay and input of every row and state element, and what the read-out needs."""
    c = s["case"]
    D, G = c["channels"], c["groups"]
    x, dt = s["x"].float(), s["dt"].float() + s["dt_bias"]
    dt = torch.nn.functional.softplus(dt)
    wide = lambda t: t.float().repeat_interleave(D // G, -2)  # noqa: E731
    a = torch.exp(dt[..., None] * -torch.exp(s["A_log"]))
    b = (dt * x)[..., None] * wide(s["B"])
    return x, a, b, wide


def _read_out(s, h, x, wide):
    y = (h * wide(s["C"])).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype)


def _plain_scan_prefill(s):
    x, a, b, wide = _steps(s)
    cu, slots = s["cu"].long(), s["slots"].long()
    full = cu[1:] > cu[:-1]
    first, last = cu[:-1][full], cu[1:][full] - 1
    h0 = s["pool"][slots] * s["has"][:, None, None]
    # a row is h -> a h + b; the first row of a sequence takes its initial state into b.
    # Rows are composed over 1, 2, 4, ... predecessors until every prefix is covered.
    b[first] += a[first] * h0[full]
    a[first] = 0
    step = 1
    while step < s["max_len"]:
        b[step:] += a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    h0[full] = b[last]
    s["pool"][slots] = h0
    return _read_out(s, b, x, wide), s["pool"]


def _plain_scan_decode(s):
    x, a, b, wide = _steps(s)
    live = s["slots"] >= 0
    slots = s["slots"].long().clamp(min=0)
    step = 1
    b[:, 0] += a[:, 0] * s["pool"][slots]
    a[:, 0] = 0
    while step < b.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    y = _read_out(s, b, x, wide)
    s["pool"][slots[live]] = b[live][:, -1]
    return torch.where(live[:, None, None], y, torch.zeros_like(y)), s["pool"]


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float()
    if s["res"] is not None:
        r = r + s["res"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * s["w"]
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * torch.sigmoid(z) * (z if c["gate"] == "silu" else 1.0)
    res = [] if s["res"] is None else [r.to(s["x"].dtype)]
    if not c["bits8"]:
        return [y.to(s["x"].dtype)] + res
    group = c["group"] or c["width"]
    pad = -c["width"] % group
    yg = torch.nn.functional.pad(y, (0, pad)).unflatten(-1, (-1, group))
    scales = yg.abs().amax(-1).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (yg / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)[..., :c["width"]]
    return [q.to(torch.float8_e4m3fn)] + res + [scales]


PLAIN = {"conv_prefill": _plain_conv_prefill, "conv_decode": _plain_conv_decode,
         "scan_prefill": _plain_scan_prefill, "scan_decode": _plain_scan_decode,
         "rms_norm": _plain_norm}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- floors
def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"].startswith(("conv", "scan")):
        rows = sum(_lens(c)) if c["op"].endswith("prefill") else c["seqs"] * c["tokens"]
    if c["op"].startswith("conv"):
        ch, W = c["channels"], c["width"]
        state = 2 * c["seqs"] * (W - 1) * ch * e
        return {"bytes": 2 * rows * ch * e + state + ch * W * 4, "flops": rows * ch * (2 * W + 4)}
    if c["op"].startswith("scan"):
        D, S, G = c["channels"], c["size"], c["groups"]
        row = (3 + c["gate"]) * D + 2 * G * S
        return {"bytes": rows * row * e + 8 * c["seqs"] * D * S + 4 * D * (S + 2),
                "flops": rows * D * (7 * S + 8)}
    n = c["tokens"] * c["heads"] * c["width"]
    moved = e * (1 + 2 * c["residual"] + (c["gate"] != "none")) + (1 if c["bits8"] else e)
    groups = -(-c["width"] // (c["group"] or c["width"])) if c["bits8"] else 0
    return {"bytes": n * moved + 4 * c["width"] + 4 * groups * c["tokens"] * c["heads"],
            "flops": n * (6 + 4 * (c["gate"] != "none") + 2 * c["bits8"])}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_conv(s, cu):
    """Sequence by sequence, tap by tap."""
    c = s["case"]
    W, x = c["width"], s["x"].double().flatten(0, -2)
    w = s["w"].double()
    y, pool = torch.zeros_like(x), s["pool"].double().clone()
    for n in range(c["seqs"]):
        slot, lo, hi = int(s["slots"][n]), cu[n], cu[n + 1]
        if slot < 0:
            continue
        past = pool[slot].clone()
        if "has" in s and not bool(s["has"][n]):
            past.zero_()
        u = torch.cat([past, x[lo:hi]])
        acc = torch.zeros_like(x[lo:hi])
        for j in range(W):
            acc += u[j:j + hi - lo] * w[:, j]
        if s["b"] is not None:
            acc += s["b"].double()
        y[lo:hi] = acc / (1 + torch.exp(-acc)) if c["silu"] else acc
        pool[slot] = u[hi - lo:]
    P = c["parts"]
    shape = s["x"].shape[:-1] + (c["channels"] // P,)
    if P == 1:
        return y.view(shape), pool
    return torch.stack([t.reshape(shape) for t in y.chunk(P, -1)]), pool


def _exact_scan(s, cu):
    """Token by token, the sequences side by side (the longest first)."""
    c = s["case"]
    D, S, G = c["channels"], c["size"], c["groups"]
    flat = lambda t, k: t.flatten(0, t.dim() - k - 1).double()  # noqa: E731
    x, dt = flat(s["x"], 1), flat(s["dt"], 1) + s["dt_bias"].double()
    dt = torch.where(dt > 30, dt, torch.log1p(torch.exp(dt.clamp(max=30))))
    B, C = flat(s["B"], 2), flat(s["C"], 2)
    A = -torch.exp(s["A_log"].double())
    y, pool = torch.zeros_like(x), s["pool"].double().clone()
    slots = s["slots"].tolist()
    has = s["has"].tolist() if "has" in s else [True] * c["seqs"]
    order = sorted((n for n in range(c["seqs"]) if slots[n] >= 0), key=lambda n: cu[n] - cu[n + 1])
    at = torch.tensor([slots[n] for n in order], device=x.device)
    h = pool[at] * torch.tensor([float(has[n]) for n in order], device=x.device,
                                dtype=torch.float64)[:, None, None]
    start = torch.tensor([cu[n] for n in order], device=x.device)
    lens = [cu[n + 1] - cu[n] for n in order]
    of = torch.arange(D, device=x.device) // (D // G)
    k = len(order)
    for p in range(max(lens, default=0)):
        while lens[k - 1] <= p:
            k -= 1
        r = start[:k] + p
        d = dt[r][..., None]
        h[:k] = torch.exp(d * A) * h[:k] + d * x[r][..., None] * B[r][:, of]
        y[r] = (h[:k] * C[r][:, of]).sum(-1)
    y += s["skip"].double() * x
    for i, n in enumerate(slots):
        if n < 0:
            y[cu[i]:cu[i + 1]] = 0
    if s["z"] is not None:
        z = flat(s["z"], 1)
        y *= z / (1 + torch.exp(-z))
    pool[at] = h
    return y.view(s["x"].shape), pool


def _exact_norm(s):
    c = s["case"]
    r = s["x"].double()
    r = r if s["res"] is None else r + s["res"].double()
    y = r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["width"] + 1e-6) * s["w"].double()
    if s["gate"] is not None:
        z = s["gate"].double()
        y *= (z if c["gate"] == "silu" else 1) / (1 + torch.exp(-z))
    res = [] if s["res"] is None else [r]
    if not c["bits8"]:
        return [y] + res
    group, q, scales = c["group"] or c["width"], torch.empty_like(y), []
    for lo in range(0, c["width"], group):
        part = y[..., lo:lo + group]
        sc = part.abs().amax(-1, keepdim=True).clamp(min=AMAX_FLOOR) / E4M3_MAX
        q[..., lo:lo + group] = part / sc
        scales.append(sc)
    return [q] + res + [torch.cat(scales, -1)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rms_norm":
        return _exact_norm(s)
    if case["op"].endswith("prefill"):
        cu = s["cu"].tolist()
    else:
        cu = [n * case["tokens"] for n in range(case["seqs"] + 1)]
    return _exact_conv(s, cu) if case["op"].startswith("conv") else _exact_scan(s, cu)
