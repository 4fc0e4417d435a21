"""Cases of the training and serving operators beside the WTConv layer: the gated scan over tokens
or pixels (forward, forward + backward, one-token step) and the AdamW update of many tensors with
the global gradient norm it clips by.

``run`` computes a case in its plain form (elementary torch operations in fp32), or, where ``own``
is true, through the package's operators.  Definitions:

  scan    z = gate + bias_c, a = sigmoid(z), h_t = a_t h_{t-1} + (1 - a_t) x_t, y_t = h_t; from
          position lengths[b] on the state stays, y is 0 and no gradient flows.
  step    the scan of one token per sequence on a pool of states: sequence b owns row slots[b];
          a sequence whose slot is -1 is idle (y = 0).
  adamw   norm = |g|_2 over all tensors, s = min(1, max_norm / (norm + 1e-6)), g' = s g,
          m' = b1 m + (1 - b1) g', v' = b2 v + (1 - b2) g'^2,
          p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps).
          In 8 bits m and v are held per block of 256 elements of a tensor: a code c and the
          block's maximum M, m = c|c| / 127^2 M (c int8), v = (c / 255)^4 M (c uint8).  A value is
          held by the code below or above it, by its place between the two and a threshold u that
          only the element's index and the step number set; a positive v never gets code 0.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256          # elements that share one maximum in the 8-bit states
K_INDEX, K_STEP = 3242174889, 2447445414   # 2^32 / p and 2^32 / p^2, p^3 = p + 1
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 37


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a few interactive sequences: a call whose latency counts
        {"name": "step_8x768_bf16", "op": "step", "B": 8, "C": 768, "slots": 8, "dtype": "bf16"},
        # a decoding step of a full serving batch on a larger pool of states, some slots idle
        {"name": "step_256x1536_f16", "op": "step", "B": 256, "C": 1536, "slots": 1024, "dtype": "f16"},
        # prefill of a ragged batch (an empty and a one-token prompt among them); x and gate are the
        # two halves of one projection's output, so their rows are strided
        {"name": "prefill_tokens_bf16", "op": "scan", "layout": "tokens", "B": 32, "T": 2048, "C": 768,
         "dtype": "bf16", "ragged": True, "h0": True, "halves": True},
        # a scan over the pixels of the 512 x 512 planes of one image: few rows, each very long
        {"name": "long_planes_bf16", "op": "scan", "layout": "planes", "B": 1, "T": 1 << 18, "C": 32,
         "dtype": "bf16", "ragged": False, "h0": False, "halves": False},
        # training on the 56 x 56 fp32 planes of the stage-1 workload
        {"name": "train_stage1_f32", "op": "train", "layout": "planes", "B": 64, "T": 3136, "C": 96,
         "dtype": "f32", "ragged": False, "h0": False, "halves": False},
        # training on the 256 x 256 bf16 planes of the high-resolution workload (the largest case)
        {"name": "train_hires_bf16", "op": "train", "layout": "planes", "B": 16, "T": 65536, "C": 64,
         "dtype": "bf16", "ragged": False, "h0": False, "halves": False},
        # training on token sequences, x and gate from one projection
        {"name": "train_tokens_bf16", "op": "train", "layout": "tokens", "B": 8, "T": 4096, "C": 1024,
         "dtype": "bf16", "ragged": False, "h0": True, "halves": True},
        # training on a small ragged batch of odd sizes: no row is aligned to a vector
        {"name": "train_tokens_odd_f16", "op": "train", "layout": "tokens", "B": 3, "T": 1001, "C": 333,
         "dtype": "f16", "ragged": True, "h0": True, "halves": False},
        # the update of the four-layer workload's parameters: twenty small tensors, latency counts
        {"name": "adamw32_four_layers", "op": "adamw", "bits": 32, "sizes": "four_layers", "n": 0, "tensors": 20,
         "grad": "f32", "copy": False},
        # the update of a backbone's parameters in mixed precision: bf16 gradients, a bf16 working copy
        {"name": "adamw32_100m_bf16", "op": "adamw", "bits": 32, "sizes": "mixed", "n": 100_000_003, "tensors": 150,
         "grad": "bf16", "copy": True},
        # the same twenty small tensors with 8-bit states
        {"name": "adamw8_four_layers", "op": "adamw", "bits": 8, "sizes": "four_layers", "n": 0, "tensors": 20,
         "grad": "f32", "copy": False},
        # a large update with 8-bit states
        {"name": "adamw8_130m_f32", "op": "adamw", "bits": 8, "sizes": "mixed", "n": 130_000_001, "tensors": 60,
         "grad": "f32", "copy": False},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step"] + ["scan"] * 2 + ["train"] * 3 + ["adamw"] * 3)
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "step":
        B = _log_uniform(rng, 1, 512)
        return {"op": op, "B": B, "C": _log_uniform(rng, 32, 4096), "slots": B + rng.randrange(0, 4 * B), "dtype": dtype}
    if op == "adamw":
        return {"op": op, "bits": rng.choice([32, 8]), "sizes": "mixed", "n": _log_uniform(rng, 5_000, 100_000_000),
                "tensors": _log_uniform(rng, 1, 300), "grad": rng.choice(["f32", "bf16", "f16"]),
                "copy": rng.random() < 0.5}
    layout = rng.choice(["tokens", "planes"])
    most = 1 << 25
    T = _log_uniform(rng, 1, 1 << 18)
    C = _log_uniform(rng, 4, min(4096, max(4, most // T)))
    B = _log_uniform(rng, 1, min(128, max(1, most // (T * C))))
    return {"op": op, "layout": layout, "B": B, "T": T, "C": C, "dtype": dtype, "ragged": rng.random() < 0.5,
            "h0": rng.random() < 0.5, "halves": layout == "tokens" and rng.random() < 0.5}


def _tensor_sizes(case):
    """Element counts of an adamw case's tensors, in order."""
    if case["sizes"] == "four_layers":
        sizes = []
        for C, L in ((96, 4), (192, 3), (384, 2), (768, 1)):
            sizes += [C * 25, C, C, L * 4 * C * 25, L * 4 * C]
        return sizes
    r = random.Random(case["n"] * 1009 + case["tensors"])
    shares = [math.exp(r.uniform(0, 6)) if r.random() < 0.6 else 0.5 for _ in range(case["tensors"])]
    return [max(1, int(case["n"] * s / sum(shares))) for s in shares]


def _layout_flat(case):
    """Offsets of the tensors in one flat buffer, each at a multiple of BLOCK, and its length."""
    offsets, end = [], 0
    for n in _tensor_sizes(case):
        offsets.append(end)
        end += -(-n // BLOCK) * BLOCK
    return offsets, end


def work(case):
    e = {"f32": 4, "bf16": 2, "f16": 2}[case.get("dtype", case.get("grad"))]
    if case["op"] == "step":
        n = case["B"] * case["C"]
        return {"bytes": n * (3 * e + 8) + 4 * case["C"] + 4 * case["B"], "flops": 12 * n}
    if case["op"] == "adamw":
        n = sum(_tensor_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8   # 8 bits: the values are returned too
        return {"bytes": n * (8 + e + state + (2 if case["copy"] else 0)), "flops": 20 * n}
    n, rows = case["B"] * case["C"] * case["T"], case["B"] * case["C"]
    if case["op"] == "scan":
        return {"bytes": 3 * n * e + 4 * rows * (1 + case["h0"]) + 4 * case["C"], "flops": 12 * n}
    return {"bytes": 8 * n * e + 4 * rows * (3 + case["h0"]) + 8 * case["C"], "flops": 42 * n}


# ------------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Lengths of a ragged batch: spread over 0..T, the first empty and the second of one token."""
    r = random.Random(seed)
    got = [r.randint(0, case["T"]) for _ in range(case["B"])]
    if case["B"] > 2:
        got[0], got[1], got[2] = 0, 1, case["T"]
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    B, C, dt = case["B"], case["C"], DTYPES[case["dtype"]]
    s = {"case": case, "bias": torch.rand(C, generator=gen, device="cuda") * 5 + 1}  # memories of 4 to 400 tokens
    if case["op"] == "step":
        s["x"], s["gate"] = normal(B, C).to(dt), normal(B, C).to(dt)
        s["pool"] = normal(case["slots"], C)
        slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        if B > 4:
            slots[B // 2] = -1
        s["slots"] = slots
        return s
    T, tokens = case["T"], case["layout"] == "tokens"
    if case["halves"]:
        both = normal(B, T, 2 * C).to(dt)
        s["x"], s["gate"] = both[:, :, :C], both[:, :, C:]
    else:
        shape = (B, T, C) if tokens else (B, C, T)
        s["x"], s["gate"] = normal(*shape).to(dt), normal(*shape).to(dt)
    s["h0"] = normal(B, C) if case["h0"] else None
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.tensor(_lengths(case, seed), dtype=torch.int32, device="cuda")
        t = torch.arange(T, device="cuda")
        padding = t[None, :] >= s["lengths"][:, None]
        padding = padding[:, :, None] if tokens else padding[:, None, :]
        s["x"].masked_fill_(padding, float("nan"))  # whatever an earlier use left there
    if case["op"] == "train":
        s["dy"] = normal(*s["x"].shape).to(dt)
        s["dh_last"] = normal(B, C)
    return s


def _quantise(x, kind, index, step):
    """8-bit codes and block maxima of a flat fp32 buffer whose tensors start at multiples of BLOCK;
    index: each element's index in its tensor."""
    x = x.view(-1, BLOCK)
    power, top = (2, 127.0) if kind == "m" else (4, 255.0)
    size = x.abs()
    most = size.amax(1, keepdim=True)
    most = torch.where(most < 2.0 ** -90, torch.zeros_like(most), most)
    y = torch.where(most > 0, size * (top ** power / most), torch.zeros_like(x))
    root = y.sqrt() if kind == "m" else y.sqrt().sqrt()
    low = root.floor().clamp_(max=top - 1)
    square, square_up = low * low, (low + 1) * (low + 1)
    level, level_up = (square, square_up) if kind == "m" else (square * square, square_up * square_up)
    code = low + (y - level > _threshold(index, step) * (level_up - level)).float()
    if kind == "v":
        code = torch.where(y > 0, code.clamp(min=1), code)
        return code.to(torch.uint8).view(-1), most.view(-1)
    return (code * torch.sign(x)).to(torch.int8).view(-1), most.view(-1)


def _threshold(index, step):
    """u = frac((i K_INDEX + step K_STEP) / 2^32), its first 24 bits."""
    return (((index.view(-1, BLOCK) * K_INDEX + step * K_STEP) & 0xFFFFFFFF) >> 8).float() * 2.0 ** -24


def _values(code, most, kind):
    """What 8-bit codes stand for, fp32."""
    c, most = code.view(-1, BLOCK).float(), most.view(-1, 1)
    if kind == "m":
        return (c * c.abs() * (most * (1.0 / 127.0 ** 2))).view(-1)
    c = c * c
    return (c * c * (most * (1.0 / 255.0 ** 4))).view(-1)


def _prepare_adamw(case, gen):
    offsets, total = _layout_flat(case)
    sizes = _tensor_sizes(case)
    index = torch.arange(total, device="cuda")
    starts = torch.tensor(offsets, device="cuda")
    which = torch.searchsorted(starts, index, right=True) - 1
    index -= starts[which]                                       # index of an element in its tensor
    used = index < torch.tensor(sizes, device="cuda")[which]

    def normal(scale):
        return torch.randn(total, generator=gen, device="cuda").mul_(scale).masked_fill_(~used, 0.0)

    # gradients of tensors differ in size, those of single elements too; the averages are as after
    # some steps of such gradients
    spread = torch.exp(torch.rand(total, generator=gen, device="cuda") * 3 - 3)
    spread *= torch.exp(-0.2 * (which % 20).float()) * 1e-2
    s = {"case": case, "index": index, "p": normal(0.05), "g": (normal(1.0) * spread).to(DTYPES[case["grad"]])}
    m = normal(0.3) * spread
    v = (spread * spread * (0.5 + torch.rand(total, generator=gen, device="cuda"))).masked_fill_(~used, 0.0)
    # a step whose gradients are clipped; with 8-bit states one that stays under the limit, as most do,
    # where the factor is exactly 1 and both sides hold the same codes
    norm = float(s["g"].double().norm())
    s["max_norm"] = norm * (0.5 if case["bits"] == 32 else 4.0)
    if case["bits"] == 8:
        s["m"], s["m_max"] = _quantise(m, "m", index, STEP - 1)
        s["v"], s["v_max"] = _quantise(v, "v", index, STEP - 1)
    else:
        s["m"], s["v"] = m, v
    s["copy"] = s["p"].to(torch.bfloat16) if case["copy"] else None
    if own:  # the optimiser object that a training program builds once over its tensors
        from memory_bound_cnn_gb300 import AdamW

        def split(flat, per=1):
            return [flat[o // per:(o // per) + -(-n // per)] for o, n in zip(offsets, sizes)]

        s["optimiser"] = AdamW(
            split(s["p"]), split(s["g"]), state_bits=case["bits"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
            weight_decay=DECAY, copies=split(s["copy"]) if case["copy"] else None, count=STEP - 1,
            states={"m": split(s["m"]), "v": split(s["v"])} if case["bits"] == 32 else
            {"m": split(s["m"]), "v": split(s["v"]), "m_max": split(s["m_max"], BLOCK), "v_max": split(s["v_max"], BLOCK)})
        s["m_values"], s["v_values"] = torch.zeros_like(s["p"]), torch.zeros_like(s["p"])
        s["m_views"], s["v_views"] = split(s["m_values"]), split(s["v_values"])
    return s


# ---------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"step": _own_step, "scan": _own_scan, "train": _own_train, "adamw": _own_adamw}[op](state)
    return {"step": _plain_step, "scan": _plain_scan, "train": _plain_train, "adamw": _plain_adamw}[op](state)


def _own_step(s):
    from memory_bound_cnn_gb300 import wtconv_scan_step

    return wtconv_scan_step(s["x"], s["gate"], s["bias"], s["pool"], slots=s["slots"]), s["pool"]


def _own_scan(s):
    from memory_bound_cnn_gb300 import wtconv_scan_forward

    y, h_last, _ = wtconv_scan_forward(s["x"], s["gate"], s["bias"], h0=s["h0"], lengths=s["lengths"],
                                       layout=s["case"]["layout"])
    return y, h_last


def _own_train(s):
    from memory_bound_cnn_gb300 import wtconv_scan_backward, wtconv_scan_forward

    layout = s["case"]["layout"]
    y, h_last, states = wtconv_scan_forward(s["x"], s["gate"], s["bias"], h0=s["h0"], lengths=s["lengths"],
                                            layout=layout, keep_states=True)
    dx, dgate, dbias, dh0 = wtconv_scan_backward(s["x"], s["gate"], s["bias"], states, s["dy"], dh_last=s["dh_last"],
                                                 lengths=s["lengths"], layout=layout)
    return y, h_last, dx, dgate, dbias, dh0


def _own_adamw(s):
    optimiser = s["optimiser"]
    clip = optimiser.grad_norm(s["max_norm"])
    optimiser.step(clip=clip, count=STEP)
    out = {"p": s["p"], "clip": clip}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if s["case"]["bits"] == 32:
        return {**out, "m": s["m"], "v": s["v"]}
    optimiser.state_values(s["m_views"], s["v_views"])
    return {**out, "m": s["m_values"], "v": s["v_values"]}


def _plain_step(s):
    slots = s["slots"].long()
    live = (slots >= 0)[:, None]
    a = torch.sigmoid(s["gate"].float() + s["bias"])
    h = a * s["pool"][slots.clamp(min=0)] + (1 - a) * s["x"].float()
    # idle sequences leave the pool alone: their rows go to one scratch row past its end
    pool = torch.cat([s["pool"], s["pool"][:1]])
    pool[torch.where(slots >= 0, slots, len(s["pool"]))] = h
    s["pool"].copy_(pool[:-1])
    return torch.where(live, h, torch.zeros_like(h)).to(s["x"].dtype), s["pool"]


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along the last axis, by doubling the span of each partial result."""
    a, u, d = a.clone(), u.clone(), 1
    while d < u.shape[-1]:
        u[..., d:] += a[..., d:] * u[..., :-d]
        a[..., d:] = a[..., d:] * a[..., :-d]
        d *= 2
    return u


def _plain_parts(s):
    """x, a, 1 - a and the mask of valid positions as (B, C, T), fp32."""
    x, gate = s["x"], s["gate"]
    if s["case"]["layout"] == "tokens":
        x, gate = x.transpose(1, 2), gate.transpose(1, 2)
    z = gate.float() + s["bias"][:, None]
    a, b, x, valid = torch.sigmoid(z), torch.sigmoid(-z), x.float(), None
    if s["lengths"] is not None:
        valid = (torch.arange(x.shape[2], device=x.device) < s["lengths"][:, None])[:, None, :]
        a, b, x = torch.where(valid, a, 1.0), torch.where(valid, b, 0.0), torch.where(valid, x, 0.0)
    return x, a, b, valid


def _plain_hidden(s, x, a, b):
    u = b * x
    if s["h0"] is not None:
        u[..., 0] += a[..., 0] * s["h0"]
    return _linear_scan(a, u)


def _back(s, t, valid):
    """A (B, C, T) result in the case's layout and type, zero past each length."""
    t = t if valid is None else torch.where(valid, t, 0.0)
    t = t.transpose(1, 2) if s["case"]["layout"] == "tokens" else t
    return t.to(s["x"].dtype)


def _plain_scan(s):
    x, a, b, valid = _plain_parts(s)
    h = _plain_hidden(s, x, a, b)
    return _back(s, h, valid), h[..., -1].clone()


def _plain_train(s):
    x, a, b, valid = _plain_parts(s)
    h = _plain_hidden(s, x, a, b)
    y, h_last = _back(s, h, valid), h[..., -1].clone()
    first = torch.zeros_like(h_last) if s["h0"] is None else s["h0"]
    before = torch.cat([first[..., None], h[..., :-1]], -1)
    dy = s["dy"].transpose(1, 2) if s["case"]["layout"] == "tokens" else s["dy"]
    dy = dy.float() if valid is None else torch.where(valid, dy.float(), 0.0)
    u = dy.flip(-1)
    u[..., 0] += s["dh_last"]
    a_next = torch.cat([torch.ones_like(a[..., :1]), a.flip(-1)[..., :-1]], -1)
    dh = _linear_scan(a_next, u).flip(-1)
    dgate = dh * (before - x) * a * b
    return y, h_last, _back(s, b * dh, valid), _back(s, dgate, valid), dgate.sum((0, 2)), a[..., 0] * dh[..., 0]


def _plain_adamw(s):
    case = s["case"]
    g = s["g"].float()
    norm = (g * g).sum().sqrt()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    g = g * scale
    small = case["bits"] == 8
    m = _values(s["m"], s["m_max"], "m") if small else s["m"]
    v = _values(s["v"], s["v_max"], "v") if small else s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    c1, c2 = 1 - BETA1 ** STEP, 1 - BETA2 ** STEP
    p = s["p"] * (1 - LR * DECAY) - (LR / c1) * (m / (v.sqrt() * (1 / math.sqrt(c2)) + EPS))
    s["p"].copy_(p)
    out = {"p": s["p"], "clip": torch.stack([norm, scale])}
    if s["copy"] is not None:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if not small:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {**out, "m": s["m"], "v": s["v"]}
    for name, x in (("m", m), ("v", v)):
        code, most = _quantise(x, name, s["index"], STEP)
        s[name].copy_(code)
        s[name + "_max"].copy_(most)
        out[name] = _values(code, most, name)
    return out


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    x, gate = s["x"].double(), s["gate"].double()
    bias = s["bias"].double()
    if case["op"] == "step":
        pool, y = s["pool"].double(), torch.zeros_like(x)
        for b, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                keep = 1 / (1 + torch.exp(-(gate[b] + bias)))
                pool[slot] = keep * pool[slot] + (1 - keep) * x[b]
                y[b] = pool[slot]
        return y, pool
    if case["T"] > 140_000 and case["op"] == "train":
        return None
    # time first, one position after the other
    order = (1, 0, 2) if case["layout"] == "tokens" else (2, 0, 1)
    x, gate = x.permute(order).contiguous(), gate.permute(order).contiguous()
    T, B, C = x.shape
    lengths = torch.full((B,), T, device=x.device) if s["lengths"] is None else s["lengths"].long()
    ends = lengths[:, None]
    forget = 1 / (1 + torch.exp(-(gate + bias)))
    h = torch.zeros(B, C, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    kept = [h] if case["op"] == "train" else None
    y = torch.zeros_like(x)
    ragged = s["lengths"] is not None
    for t in range(T):
        new = torch.lerp(x[t], h, forget[t])
        if ragged:
            new = torch.where(t < ends, new, h)
            y[t] = torch.where(t < ends, new, 0.0)
        else:
            y[t] = new
        h = new
        if kept is not None:
            kept.append(h)
    back = (1, 0, 2) if case["layout"] == "tokens" else (1, 2, 0)
    if case["op"] == "scan":
        return y.permute(back).contiguous(), h
    dy = s["dy"].double().permute(order).contiguous()
    flow = s["dh_last"].double()
    dx, dgate = torch.zeros_like(x), torch.zeros_like(x)
    for t in reversed(range(T)):
        a = forget[t]
        total = flow + dy[t]
        one, two, new = total * (1 - a), total * (kept[t] - x[t]) * a * (1 - a), total * a
        if ragged:
            live = t < ends
            dx[t], dgate[t] = torch.where(live, one, 0.0), torch.where(live, two, 0.0)
            flow = torch.where(live, new, flow)
        else:
            dx[t], dgate[t], flow = one, two, new
    return (y.permute(back).contiguous(), h, dx.permute(back).contiguous(), dgate.permute(back).contiguous(),
            dgate.sum((0, 1)), flow)


def _exact_adamw(s):
    case = s["case"]
    g, p = s["g"].double(), s["p"].double()
    norm = g.norm()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    g = g * scale

    def held(code, most, top, power):
        c = code.double().view(-1, BLOCK)
        return ((c.abs() / top) ** power * torch.sign(c) * most.double()[:, None]).view(-1)

    small = case["bits"] == 8
    m = held(s["m"], s["m_max"], 127, 2) if small else s["m"].double()
    v = held(s["v"], s["v_max"], 255, 4) if small else s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    rate = LR / (1 - BETA1 ** STEP)
    p = p - LR * DECAY * p - rate * m / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
    out = {"p": p, "clip": torch.stack([norm, scale])}
    if case["copy"]:
        out["copy"] = p
    if not small:
        return {**out, "m": m, "v": v}
    for name, x, top, power in (("m", m, 127, 2), ("v", v, 255, 4)):
        x = x.view(-1, BLOCK)
        most = x.abs().amax(1, keepdim=True)
        share = torch.where(most > 0, x.abs() / most, 0.0)
        low = torch.floor(share ** (1 / power) * top).clamp(max=top - 1)
        below, above = (low / top) ** power, ((low + 1) / top) ** power
        place = ((s["index"] * K_INDEX + STEP * K_STEP) % 2 ** 32).view(-1, BLOCK).double() / 2 ** 32
        up = share - below > torch.floor(place * 2 ** 24) / 2 ** 24 * (above - below)
        if name == "v":
            up |= (low == 0) & (share > 0)
        out[name] = (torch.where(up, above, below) * torch.sign(x) * most).view(-1)
    return out
