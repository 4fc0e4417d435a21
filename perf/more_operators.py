"""Cases of a selective state space scan with the short causal convolution and the root-mean-square norm
around it: forward, forward + backward, and the one-token forms of serving.

``run`` computes a case in its plain form (elementary torch operations in fp32), or, where ``own``
is true, through the package's operators.  Definitions:

  scan    d = softplus(dt + dt_bias_c) (or dt as it is), a_tn = exp(d_t A_cn),
          h_tn = a_tn h_{t-1,n} + d_t x_t B_tn,  y_t = (sum_n C_tn h_tn + D_c x_t) silu(z_t)
          for every channel c with its N states; B and C belong to the channels of a group.
  conv    y_t = silu(bias_c + sum_k w_ck x_{t-K+1+k}); a state holds the K-1 inputs before the first
          position, and the last state those before the position after the last.
  norm    total = x + residual, rounded to the residual's type; y = total rsqrt(mean total^2 + eps) w,
          or y in e4m3 by blocks of a row: scale = max |y| / 448, q = y / scale rounded.
  From position lengths[b] on, outputs and gradients are 0 and states stay.  A one-token step works on
  a pool of states: sequence b owns slots[b], a slot of -1 is idle (y = 0).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
MOST = 1 << 28     # states times positions of a drawn scan


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a few interactive sequences: a call whose latency counts
        {"name": "scan_step_8x768_bf16", "op": "scan_step", "B": 8, "C": 768, "N": 16, "G": 1, "slots": 8, "dtype": "bf16"},
        # prefill of a ragged batch (an empty and a one-token prompt among them); x and z are the halves of
        # one projection's output, B and C those of another, so that all rows are strided
        {"name": "scan_prefill_bf16", "op": "scan", "layout": "tokens", "B": 16, "T": 2048, "C": 768, "N": 16, "G": 1,
         "dtype": "bf16", "ragged": True, "h0": True, "z": True, "D": True, "softplus": True, "halves": True},
        # a scan over the pixels of one image's 256 x 256 planes: few channels, each sequence very long
        {"name": "scan_pixels_bf16", "op": "scan", "layout": "planes", "B": 1, "T": 65536, "C": 64, "N": 16, "G": 1,
         "dtype": "bf16", "ragged": False, "h0": False, "z": False, "D": True, "softplus": True, "halves": False},
        # training on the 56 x 56 fp32 planes of the stage-1 workload, few states
        {"name": "scan_train_stage1_f32", "op": "scan_train", "layout": "planes", "B": 64, "T": 3136, "C": 96, "N": 8, "G": 1,
         "dtype": "f32", "ragged": False, "h0": False, "z": True, "D": True, "softplus": True, "halves": False},
        # training on token sequences (the largest case)
        {"name": "scan_train_tokens_bf16", "op": "scan_train", "layout": "tokens", "B": 8, "T": 4096, "C": 1024, "N": 16, "G": 1,
         "dtype": "bf16", "ragged": False, "h0": False, "z": True, "D": True, "softplus": True, "halves": True},
        # training on a small ragged batch of odd sizes, three groups of channels: no row is aligned to a vector
        {"name": "scan_train_odd_f16", "op": "scan_train", "layout": "tokens", "B": 3, "T": 1001, "C": 333, "N": 13, "G": 3,
         "dtype": "f16", "ragged": True, "h0": True, "z": True, "D": True, "softplus": True, "halves": False},
        # a decoding step of a full serving batch on a larger pool of states, some slots idle
        {"name": "conv_step_256x2048_f16", "op": "conv_step", "B": 256, "C": 2048, "K": 4, "slots": 1024, "dtype": "f16", "silu": True},
        # training on token sequences
        {"name": "conv_train_tokens_bf16", "op": "conv_train", "layout": "tokens", "B": 8, "T": 4096, "C": 2048, "K": 4,
         "dtype": "bf16", "ragged": False, "state": False, "silu": True, "halves": True},
        # training on ragged pixel sequences of an odd number of fp32 channels
        {"name": "conv_train_planes_f32", "op": "conv_train", "layout": "planes", "B": 32, "T": 3136, "C": 97, "K": 3,
         "dtype": "f32", "ragged": True, "state": True, "silu": True, "halves": False},
        # the norm before an 8-bit projection in a decoding step: a call whose latency counts
        {"name": "norm8_step_8x768_bf16", "op": "norm8", "rows": 8, "C": 768, "block": 0, "dtype": "bf16", "residual": "bf16"},
        # the same for a long prompt, a scale for every 128 values, the residual kept in fp32
        {"name": "norm8_prefill_bf16", "op": "norm8", "rows": 16384, "C": 2048, "block": 128, "dtype": "bf16", "residual": "f32"},
        # training on token sequences
        {"name": "norm_train_tokens_bf16", "op": "norm_train", "rows": 32768, "C": 1024, "dtype": "bf16", "residual": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan_step", "scan", "scan", "scan_train", "scan_train", "conv_step", "conv_train", "conv_train",
                     "norm8", "norm_train"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    chance = rng.random
    if op in ("norm8", "norm_train"):
        C = _log_uniform(rng, 32, 8192)
        case = {"op": op, "rows": _log_uniform(rng, 1, min(65536, (1 << 25) // C)), "C": C, "dtype": dtype,
                "residual": rng.choice([dtype, "f32", "none"])}
        return {**case, "block": rng.choice([0, 128])} if op == "norm8" else case
    if op == "conv_step":
        B = _log_uniform(rng, 1, 512)
        return {"op": op, "B": B, "C": _log_uniform(rng, 32, 4096), "K": rng.choice([2, 3, 4]), "slots": B + rng.randrange(0, 4 * B),
                "dtype": dtype, "silu": chance() < 0.8}
    N, G = rng.choice([16, 16, 8, 32, 64, rng.randint(1, 64)]), rng.choice([1, 1, 2, 3])
    if op == "scan_step":
        B = _log_uniform(rng, 1, 512)
        return {"op": op, "B": B, "C": G * _log_uniform(rng, 16, 1024), "N": N, "G": G, "slots": B + rng.randrange(0, 2 * B),
                "dtype": dtype}
    layout = rng.choice(["tokens", "planes"])
    most = 1 << 25 if op == "conv_train" else MOST // N
    T = _log_uniform(rng, 1, 1 << 16)
    C = _log_uniform(rng, 4, min(2048, max(4, most // T)))
    B = _log_uniform(rng, 1, min(64, max(1, most // (T * C))))
    case = {"op": op, "layout": layout, "B": B, "T": T, "C": C, "dtype": dtype, "ragged": chance() < 0.5, "halves": chance() < 0.5}
    if op == "conv_train":
        return {**case, "K": rng.choice([2, 3, 4]), "state": chance() < 0.5, "silu": chance() < 0.8}
    return {**case, "C": G * max(1, C // G), "N": N, "G": G, "h0": chance() < 0.5, "z": chance() < 0.7, "D": chance() < 0.7,
            "softplus": chance() < 0.8}


def work(case):
    e, op = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]], case["op"]
    C = case["C"]
    if op in ("norm8", "norm_train"):
        n, r = case["rows"] * C, {"none": 0, "f32": 4, "bf16": 2, "f16": 2}[case["residual"]]
        if op == "norm8":
            return {"bytes": n * (e + 2 * r + 1) + 4 * case["rows"] * (-(-C // case["block"]) if case["block"] else 1) + 4 * C,
                    "flops": 8 * n}
        # forward: x and residual in, total and y out; backward: dy, the total and its gradient in, gradients out
        # (the total and its gradient are x and dx where there is no residual)
        both = (3 * r + (e if r != e else 0)) if r else 2 * e
        return {"bytes": n * (2 * e + 2 * r + e + both) + 8 * C, "flops": 18 * n}
    B = case["B"]
    if op == "conv_step":
        return {"bytes": B * C * e * (2 + 2 * (case["K"] - 1)) + 4 * C * (case["K"] + 1) + 4 * B, "flops": B * C * (2 * case["K"] + 5)}
    if op == "scan_step":
        N, G = case["N"], case["G"]
        return {"bytes": B * C * (4 * e + 8 * N) + 2 * B * G * N * e + 4 * C * (N + 2) + 4 * B, "flops": B * C * (7 * N + 15)}
    n = B * C * case["T"]
    if op == "conv_train":
        K = case["K"]
        return {"bytes": n * 5 * e + 8 * C * (K + 1) + B * C * (K - 1) * e * (2 + 2 * case["state"]),
                "flops": n * (8 * K + 16)}
    N, z = case["N"], case["z"]
    bc = 2 * B * case["T"] * case["G"] * N * e
    small = 4 * C * (N + 2) + 4 * B * C * N * (1 + case["h0"])
    if op == "scan":
        return {"bytes": n * e * (3 + z) + bc + small, "flops": n * (7 * N + 15)}
    return {"bytes": n * e * (8 + 3 * z) + 3 * bc + 3 * small, "flops": n * (29 * N + 50)}


# ------------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Lengths of a ragged batch: spread over 0..T, the first empty and the second of one token."""
    r = random.Random(seed)
    got = [r.randint(0, case["T"]) for _ in range(case["B"])]
    if case["B"] > 2:
        got[0], got[1], got[2] = 0, 1, case["T"]
    return got


def _slots(case, gen):
    slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:case["B"]].to(torch.int32)
    if case["B"] > 4:
        slots[case["B"] // 2] = -1
    return slots


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dt, op, C = DTYPES[case["dtype"]], case["op"], case["C"]
    s = {"case": case}
    if op in ("norm8", "norm_train"):
        rows = case["rows"]
        # channels of a residual stream differ in size, a few of them by much
        size = torch.exp(normal(C)) * torch.where(uniform(C) < 0.01, 10.0, 1.0)
        s["x"], s["weight"] = normal(rows, C).to(dt), 1 + 0.2 * normal(C)
        s["residual"] = None
        if case["residual"] != "none":
            s["residual"] = (normal(rows, C) * size).to(DTYPES[case["residual"]])
        if op == "norm_train":
            s["dy"] = normal(rows, C).to(dt)
            # what flows into the total past the norm, along the residual stream
            s["d_total"] = None if s["residual"] is None else normal(rows, C).to(s["residual"].dtype)
        return s
    B = case["B"]
    if op in ("conv_step", "conv_train"):
        K = case["K"]
        s["weight"], s["bias"] = normal(C, K) / math.sqrt(K), 0.1 * normal(C)
        if op == "conv_step":
            s["x"], s["pool"], s["slots"] = normal(B, C).to(dt), normal(case["slots"], C, K - 1).to(dt), _slots(case, gen)
            return s
    else:
        N, G = case["N"], case["G"]
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * normal(C, N))
        step = torch.exp(uniform(C) * math.log(100.0)) * 1e-3       # steps of 0.001 to 0.1: memories of 10 to 1000 tokens
        s["D"] = 1 + 0.2 * normal(C)
        s["dt_bias"] = torch.log(torch.expm1(step))
        if op == "scan_step":
            s["x"], s["z"], s["dt"] = normal(B, C).to(dt), normal(B, C).to(dt), normal(B, C).to(dt)
            s["B"], s["C"] = normal(B, G, N).to(dt), normal(B, G, N).to(dt)
            s["pool"], s["slots"] = normal(case["slots"], C, N), _slots(case, gen)
            return s
    T, tokens = case["T"], case["layout"] == "tokens"

    def pair(*inner):
        """Two activations, the halves of one tensor where the case says so."""
        n = 1
        for i in inner:
            n *= i
        axis = 2 if tokens else 1
        if case["halves"]:
            whole = normal(B, T, 2 * n) if tokens else normal(B, 2 * n, T)
            parts = whole.to(dt).chunk(2, axis)
        else:
            parts = [(normal(B, T, n) if tokens else normal(B, n, T)).to(dt) for _ in range(2)]
        if len(inner) == 1:
            return parts
        return [p.unflatten(axis, inner) for p in parts]

    if op == "conv_train":
        s["x"], _ = pair(C)
        s["dy"], _ = pair(C)
        s["state"] = normal(B, C, K - 1).to(dt) if case["state"] else None
        s["d_last"] = normal(B, C, K - 1).to(dt)
        padded = ("x", "dy")
    else:
        s["x"], s["z"] = pair(C)
        s["B"], s["C"] = pair(G, N)
        s["dt"] = normal(*s["x"].shape).to(dt)
        if not case["softplus"]:   # the steps themselves
            s["dt"] = (torch.exp(0.3 * s["dt"].float()) * (step if tokens else step[:, None])).to(dt)
            s["dt_bias"] = None
        s["h0"] = normal(B, C, N) if case["h0"] else None
        s["z"] = s["z"] if case["z"] else None
        s["D"] = s["D"] if case["D"] else None
        padded = ("x", "z", "B", "C", "dt")
        if op == "scan_train":
            s["dy"], s["dh_last"] = normal(*s["x"].shape).to(dt), normal(B, C, N)
            padded += ("dy",)
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.tensor(_lengths(case, seed), dtype=torch.int32, device="cuda")
        past = torch.arange(T, device="cuda")[None, :] >= s["lengths"][:, None]
        for k in padded:
            if s[k] is not None:
                shape = [B] + [1] * (s[k].dim() - 1)
                shape[1 if tokens else -1] = T
                s[k].masked_fill_(past.view(shape), float("nan"))  # whatever an earlier use left there
    return s


# ---------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"scan_step": _own_scan_step, "scan": _own_scan, "scan_train": _own_scan_train, "conv_step": _own_conv_step,
                "conv_train": _own_conv_train, "norm8": _own_norm8, "norm_train": _own_norm_train}[op](state)
    return {"scan_step": _plain_scan_step, "scan": _plain_scan, "scan_train": _plain_scan_train, "conv_step": _plain_conv_step,
            "conv_train": _plain_conv_train, "norm8": _plain_norm8, "norm_train": _plain_norm_train}[op](state)


def _own_scan_step(s):
    from memory_bound_cnn_gb300 import wtconv_selective_step

    y = wtconv_selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                              slots=s["slots"])
    return y, s["pool"]


def _own_scan(s):
    from memory_bound_cnn_gb300 import wtconv_selective_forward

    y, h_last, _ = wtconv_selective_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                            h0=s["h0"], lengths=s["lengths"], layout=s["case"]["layout"],
                                            softplus=s["case"]["softplus"])
    return y, h_last


def _own_scan_train(s):
    from memory_bound_cnn_gb300 import wtconv_selective_backward, wtconv_selective_forward

    inputs = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "lengths": s["lengths"], "layout": s["case"]["layout"],
            "softplus": s["case"]["softplus"]}
    y, h_last, states = wtconv_selective_forward(*inputs, h0=s["h0"], keep_states=True, **more)
    return y, h_last, *wtconv_selective_backward(*inputs, states, s["dy"], dh_last=s["dh_last"], **more)


def _own_conv_step(s):
    from memory_bound_cnn_gb300 import wtconv_causal_step

    return wtconv_causal_step(s["x"], s["weight"], s["pool"], bias=s["bias"], slots=s["slots"], silu=s["case"]["silu"]), s["pool"]


def _own_conv_train(s):
    from memory_bound_cnn_gb300 import wtconv_causal_backward, wtconv_causal_forward

    more = {"bias": s["bias"], "state": s["state"], "lengths": s["lengths"], "layout": s["case"]["layout"], "silu": s["case"]["silu"]}
    y, last = wtconv_causal_forward(s["x"], s["weight"], **more)
    return y, last, *wtconv_causal_backward(s["x"], s["weight"], s["dy"], d_last=s["d_last"], **more)


def _own_norm8(s):
    from memory_bound_cnn_gb300 import wtconv_rms_forward_e4m3

    return wtconv_rms_forward_e4m3(s["x"], s["weight"], residual=s["residual"], eps=EPS, block=s["case"]["block"])


def _own_norm_train(s):
    from memory_bound_cnn_gb300 import wtconv_rms_backward, wtconv_rms_forward

    y, total, rstd = wtconv_rms_forward(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    added = s["residual"] is not None
    dx, d_residual, d_weight = wtconv_rms_backward(s["dy"], total, s["weight"], rstd, d_total=s["d_total"], residual=added)
    return y, total if added else None, dx, d_residual, d_weight


# ------------------------------------------------------------------------------- plain forms

def _silu(z):
    return z * torch.sigmoid(z)


def _silu_slope(z):
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _into_pool(s, new, live, slots):
    """Rows of the pool replaced; idle sequences write to a scratch row past its end."""
    pool = torch.cat([s["pool"], s["pool"][:1]])
    pool[torch.where(live, slots, len(s["pool"]))] = new
    s["pool"].copy_(pool[:-1])


def _plain_scan_step(s):
    slots = s["slots"].long()
    live = slots >= 0
    x, z, (B, C) = s["x"].float(), s["z"].float(), s["x"].shape
    d = _softplus(s["dt"].float() + s["dt_bias"])
    G = s["case"]["G"]
    b, c = (s[k].float().repeat_interleave(C // G, 1) for k in ("B", "C"))
    h = torch.exp(d[..., None] * s["A"]) * s["pool"][slots.clamp(min=0)] + (d * x)[..., None] * b
    y = ((h * c).sum(-1) + s["D"] * x) * _silu(z)
    _into_pool(s, h, live, slots)
    return torch.where(live[:, None], y, 0.0).to(s["x"].dtype), s["pool"]


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1, by doubling the span of each partial result (in place)."""
    d = 1
    while d < u.shape[1]:
        u[:, d:] += a[:, d:] * u[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return u


def _valid(s):
    """The mask of valid positions (B, T), or None."""
    if s["lengths"] is None:
        return None
    return torch.arange(s["case"]["T"], device=s["x"].device) < s["lengths"][:, None]


def _time(s, name, valid):
    """An activation as (B, T, channels), (B, T, G, N) for B and C; fp32, 0 past each length."""
    t = s[name].float()
    if s["case"]["layout"] == "planes":
        t = t.movedim(-1, 1)
    return t if valid is None else torch.where(valid.view(valid.shape + (1,) * (t.dim() - 2)), t, 0.0)


def _back(s, t, valid):
    """A (B, T, ...) result in the case's layout and type, 0 past each length."""
    t = t if valid is None else torch.where(valid.view(valid.shape + (1,) * (t.dim() - 2)), t, 0.0)
    t = t.movedim(1, -1) if s["case"]["layout"] == "planes" else t
    return t.to(s["x"].dtype).contiguous()


def _scan_parts(s):
    """What both directions need: masked inputs, steps, decays and states (B, T, C, N)."""
    valid = _valid(s)
    p = {"valid": valid, "x": _time(s, "x", valid), "raw": _time(s, "dt", valid)}
    heads = p["x"].shape[2] // s["case"]["G"]
    p["B"], p["C"] = (_time(s, k, valid).repeat_interleave(heads, 2) for k in ("B", "C"))
    p["d"] = p["raw"] if s["dt_bias"] is None else _softplus(p["raw"] + s["dt_bias"])
    if valid is not None:
        p["d"] = torch.where(valid[..., None], p["d"], 0.0)
    p["a"] = torch.exp(p["d"][..., None] * s["A"])
    u = (p["d"] * p["x"])[..., None] * p["B"]
    if s["h0"] is not None:
        u[:, 0] += p["a"][:, 0] * s["h0"]
    p["h"] = _linear_scan(p["a"].clone(), u)
    p["sum"] = (p["h"] * p["C"]).sum(-1)
    if s["D"] is not None:
        p["sum"] += s["D"] * p["x"]
    return p


def _scan_y(s, p):
    y = p["sum"]
    if s["z"] is not None:
        y = y * _silu(_time(s, "z", p["valid"]))
    return _back(s, y, p["valid"])


def _plain_scan(s):
    p = _scan_parts(s)
    return _scan_y(s, p), p["h"][:, -1].clone()


def _plain_scan_train(s):
    p = _scan_parts(s)
    y, h_last, valid = _scan_y(s, p), p["h"][:, -1].clone(), p["valid"]
    dy = _time(s, "dy", valid)
    dz = None
    if s["z"] is not None:
        z = _time(s, "z", valid)
        dz = _back(s, dy * p["sum"] * _silu_slope(z), valid)
        dy = dy * _silu(z)
    # dh_t = dy_t C_t + a_{t+1} dh_{t+1}, from the end; what flows into h_last enters at the last position
    u = (dy[..., None] * p["C"]).flip(1)
    u[:, 0] += s["dh_last"]
    a_next = torch.cat([torch.ones_like(p["a"][:, :1]), p["a"].flip(1)[:, :-1]], 1)
    dh = _linear_scan(a_next, u).flip(1)
    del u, a_next
    G, (B, T, C, N) = s["case"]["G"], dh.shape
    dC = _back(s, (dy[..., None] * p["h"]).view(B, T, G, C // G, N).sum(3), valid)
    dB = _back(s, (dh * (p["d"] * p["x"])[..., None]).view(B, T, G, C // G, N).sum(3), valid)
    first = torch.zeros_like(h_last) if s["h0"] is None else s["h0"]
    through = dh * p["a"]
    dh0 = through[:, 0].clone()
    through *= torch.cat([first[:, None], p["h"][:, :-1]], 1)
    dA = (through * p["d"][..., None]).sum((0, 1))
    into = (dh * p["B"]).sum(-1)
    dd = (through * s["A"]).sum(-1) + into * p["x"]
    dx = into * p["d"]
    dD = None
    if s["D"] is not None:
        dx, dD = dx + dy * s["D"], (dy * p["x"]).sum((0, 1))
    d_bias = None
    if s["dt_bias"] is not None:
        dd = dd * torch.sigmoid(p["raw"] + s["dt_bias"])
        dd = dd if valid is None else torch.where(valid[..., None], dd, 0.0)
        d_bias = dd.sum((0, 1))
    return y, h_last, _back(s, dx, valid), _back(s, dd, valid), dA, dB, dC, dD, dz, d_bias, dh0


def _plain_conv_step(s):
    slots = s["slots"].long()
    live = slots >= 0
    window = torch.cat([s["pool"][slots.clamp(min=0)], s["x"][..., None]], -1)
    pre = (window.float() * s["weight"]).sum(-1) + s["bias"]
    y = _silu(pre) if s["case"]["silu"] else pre
    _into_pool(s, window[..., 1:], live, slots)
    return torch.where(live[:, None], y, 0.0).to(s["x"].dtype), s["pool"]


def _plain_conv_train(s):
    case, valid = s["case"], _valid(s)
    K = case["K"]
    x, dy = (_time(s, k, valid).transpose(1, 2) for k in ("x", "dy"))     # (B, C, T)
    before = torch.zeros_like(x[..., :1]).expand(-1, -1, K - 1) if s["state"] is None else s["state"].float()
    x = torch.cat([before, x], -1)
    windows = x.unfold(2, K, 1)
    pre = (windows * s["weight"][:, None]).sum(-1) + s["bias"][:, None]
    y = _silu(pre) if case["silu"] else pre
    ends = torch.full_like(x[:, 0, 0], case["T"]).long() if valid is None else s["lengths"].long()
    at = (ends[:, None] + torch.arange(K - 1, device=x.device))[:, None].expand(-1, x.shape[1], -1)
    last = x.gather(2, at).to(s["x"].dtype)
    slope = dy * _silu_slope(pre) if case["silu"] else dy
    d_weight, d_bias = (windows * slope[..., None]).sum((0, 2)), slope.sum((0, 2))
    # an input at place i of [state, x] reaches the outputs i - K + 1 to i, and the last state
    nothing = slope.new_zeros(*slope.shape[:2], K - 1)
    around = torch.cat([nothing, slope, nothing], -1)
    dx = (around.unfold(2, K, 1) * s["weight"].flip(1)[:, None]).sum(-1)
    dx = dx.scatter_add(2, at, s["d_last"].float())
    d_state = None if s["state"] is None else dx[..., :K - 1].to(s["x"].dtype)
    dx = dx[..., K - 1:].transpose(1, 2)
    return _back(s, y.transpose(1, 2), valid), last, _back(s, dx, valid), d_weight, d_bias, d_state


def _total(s):
    return s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)


def _plain_norm8(s):
    total = _total(s)
    t = total.float()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["weight"]
    rows, C = y.shape
    block = s["case"]["block"] or C
    blocks = -(-C // block)
    y = torch.nn.functional.pad(y, (0, blocks * block - C)).view(rows, blocks, block)
    scales = y.abs().amax(2) / 448
    q = (y / torch.where(scales > 0, scales, 1.0)[..., None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :C].contiguous(), scales, None if s["residual"] is None else total


def _plain_norm_train(s):
    total = _total(s)
    t, dy = total.float(), s["dy"].float()
    rstd = torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    n = t * rstd
    g = dy * s["weight"]
    d = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if s["d_total"] is not None:
        d = d + s["d_total"].float()
    none = s["residual"] is None
    return ((n * s["weight"]).to(s["x"].dtype), None if none else total, d.to(s["x"].dtype),
            None if none else d.to(s["residual"].dtype), (dy * n).sum(0))


# --------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm8", "norm_train"):
        return _exact_norm(s)
    if op in ("conv_step", "scan_step"):
        return _exact_step(s)
    return _exact_conv(s) if op == "conv_train" else _exact_scan(s)


def _exact_step(s):
    case, w = s["case"], {k: v.double() for k, v in s.items() if k not in ("case", "slots")}
    pool, y = w["pool"], torch.zeros_like(w["x"])
    for b, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        if case["op"] == "conv_step":
            seen = torch.cat([pool[slot], w["x"][b][:, None]], 1)
            pool[slot] = seen[:, 1:]
            y[b] = torch.einsum("ck,ck->c", seen, w["weight"]) + w["bias"]
            if case["silu"]:
                y[b] /= 1 + torch.exp(-y[b])
            continue
        step = torch.log(1 + torch.exp(w["dt"][b] + w["dt_bias"]))
        mine = torch.arange(case["C"], device=y.device) // (case["C"] // case["G"])
        pool[slot] *= torch.exp(step[:, None] * w["A"])
        pool[slot] += step[:, None] * w["x"][b][:, None] * w["B"][b][mine]
        y[b] = torch.einsum("cn,cn->c", pool[slot], w["C"][b][mine]) + w["D"] * w["x"][b]
        y[b] *= w["z"][b] / (1 + torch.exp(-w["z"][b]))
    return y, pool


def _time_first(s, name):
    """(T, B, ...) in 64 bits, 0 past each length."""
    t = s[name].double()
    t = t.movedim(1 if s["case"]["layout"] == "tokens" else -1, 0).contiguous()
    if s["lengths"] is not None:
        for b, n in enumerate(s["lengths"].tolist()):
            t[n:, b] = 0
    return t


def _laid_out(s, t):
    return t.movedim(0, 1 if s["case"]["layout"] == "tokens" else -1).contiguous()


def _exact_conv(s):
    case = s["case"]
    K, T, B, C = case["K"], case["T"], case["B"], case["C"]
    w, x, dy = s["weight"].double(), _time_first(s, "x"), _time_first(s, "dy")
    state = torch.zeros(K - 1, B, C, dtype=torch.float64, device=x.device)
    if s["state"] is not None:
        state = s["state"].double().permute(2, 0, 1).contiguous()
    seen = torch.cat([state, x])
    pre = s["bias"].double().expand(T, B, C).clone()
    for k in range(K):
        pre += w[:, k] * seen[k:k + T]
    gate = 1 / (1 + torch.exp(-pre)) if case["silu"] else torch.ones_like(pre)
    y = pre * gate if case["silu"] else pre.clone()
    d = dy * (gate + pre * gate * (1 - gate)) if case["silu"] else dy
    ends = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    d_seen, d_weight = torch.zeros_like(seen), torch.zeros_like(w)
    for k in range(K):
        d_seen[k:k + T] += w[:, k] * d
        d_weight[:, k] = (d * seen[k:k + T]).sum((0, 1))
    last = torch.zeros(B, C, K - 1, dtype=torch.float64, device=x.device)
    for b, n in enumerate(ends):
        last[b] = seen[n:n + K - 1, b].T
        d_seen[n:n + K - 1, b] += s["d_last"][b].double().T
        y[n:, b] = 0
    dx = d_seen[K - 1:].clone()
    for b, n in enumerate(ends):
        dx[n:, b] = 0
    return (_laid_out(s, y), last, _laid_out(s, dx), d_weight, d.sum((0, 1)),
            None if s["state"] is None else d_seen[:K - 1].permute(1, 2, 0).contiguous())


def _exact_scan(s):
    case = s["case"]
    T, B, C, N, G = case["T"], case["B"], case["C"], case["N"], case["G"]
    if T * B * C * N > 1 << 29:
        return None
    x, raw, A = _time_first(s, "x"), _time_first(s, "dt"), s["A"].double()
    mine = torch.arange(C, device=x.device) // (C // G)
    b, c = _time_first(s, "B"), _time_first(s, "C")
    step, slope = raw, torch.ones_like(raw)
    if s["dt_bias"] is not None:
        e = torch.exp(raw + s["dt_bias"].double())
        step, slope = torch.log1p(e), e / (1 + e)
    if s["lengths"] is not None:
        for i, n in enumerate(s["lengths"].tolist()):
            step[n:, i], slope[n:, i] = 0, 0
    decay = torch.exp(step[..., None] * A)
    h = torch.zeros(B, C, N, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    states = torch.empty(T + 1, B, C, N, dtype=torch.float64, device=x.device)
    states[0] = h
    driven = step * x
    for t in range(T):
        h = torch.addcmul(driven[t][..., None] * b[t][:, mine], decay[t], h)
        states[t + 1] = h
    out = torch.empty_like(x)
    per = max(1, (1 << 26) // (B * C * N))
    for t in range(0, T, per):
        out[t:t + per] = torch.einsum("tbcn,tbcn->tbc", states[t + 1:t + 1 + per], c[t:t + per][:, :, mine])
    if s["D"] is not None:
        out += s["D"].double() * x
    z = None if s["z"] is None else _time_first(s, "z")
    gate = None if z is None else 1 / (1 + torch.exp(-z))
    y = out if z is None else out * z * gate
    if case["op"] == "scan":
        return _laid_out(s, y), h
    dy = _time_first(s, "dy")
    dz = None if z is None else dy * out * (gate + z * gate * (1 - gate))
    dy = dy if z is None else dy * z * gate
    flow = s["dh_last"].double()
    d_step, d_driven, dA = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(A)
    dB, dC = torch.zeros_like(b), torch.zeros_like(c)
    for t in reversed(range(T)):
        flow = torch.addcmul(flow, dy[t][..., None], c[t][:, mine])
        dC[t] = (dy[t][..., None] * states[t + 1]).view(B, G, C // G, N).sum(2)
        dB[t] = (driven[t][..., None] * flow).view(B, G, C // G, N).sum(2)
        d_driven[t] = (flow * b[t][:, mine]).sum(-1)
        flow = flow * decay[t]
        through = flow * states[t]
        d_step[t] = (through * A).sum(-1)
        dA += (through * step[t][..., None]).sum(0)
    d_step += d_driven * x
    dx, dD = d_driven * step, None
    if s["D"] is not None:
        dx, dD = dx + dy * s["D"].double(), (dy * x).sum((0, 1))
    d_raw = d_step * slope
    if s["lengths"] is not None:
        for i, n in enumerate(s["lengths"].tolist()):
            d_raw[n:, i] = 0
    return (_laid_out(s, y), h, _laid_out(s, dx), _laid_out(s, d_raw), dA, _laid_out(s, dB), _laid_out(s, dC), dD,
            None if dz is None else _laid_out(s, dz), None if s["dt_bias"] is None else d_raw.sum((0, 1)), flow)


def _exact_norm(s):
    case, x, w = s["case"], s["x"].double(), s["weight"].double()
    total = x if s["residual"] is None else (x + s["residual"].double()).to(s["residual"].dtype).double()
    C = x.shape[1]
    size = torch.sqrt((total ** 2).sum(1, keepdim=True) / C + EPS)
    n = total / size
    kept = None if s["residual"] is None else total
    if case["op"] == "norm8":
        y, q, scales = n * w, torch.zeros_like(x), []
        block = case["block"] or C
        for at in range(0, C, block):
            part = y[:, at:at + block]
            most = part.abs().max(1, keepdim=True).values / 448
            scales.append(most)
            q[:, at:at + block] = torch.where(most > 0, part / most, 0.0).to(torch.float8_e4m3fn).double()
        return q, torch.cat(scales, 1), kept
    dy = s["dy"].double()
    d = (dy * w - n * ((dy * w * n).sum(1, keepdim=True) / C)) / size
    if s["d_total"] is not None:
        d = d + s["d_total"].double()
    return n * w, kept, d, None if kept is None else d, (dy * n).sum(0)
