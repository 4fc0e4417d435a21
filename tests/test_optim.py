"""AdamW over many tensors and the gradient norm (include/wtconv_optim.h) against their definitions."""
import ctypes

import adamw_reference as R
import numpy as np
import pytest
import torch

from memory_bound_cnn_gb300 import optim as O
from memory_bound_cnn_gb300 import wtconv as W

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# fp32 products, one square root and one quotient, each off by 2^-24 or a few: 1e-6 of the terms
BOUND = 1e-6
# (sizes of the tensors; odd starts put tensors off every vector boundary)
LISTS = {
    "one": [1], "small": [3, 1, 7, 255, 256, 257], "layer": [2400, 96, 96, 38400, 1536],
    "chunks": [2047, 2048, 2049, 5000, 0, 12345], "many": [(i * 37) % 700 for i in range(1000)],
}


def make(sizes, grad_dtype=torch.float32, bits=32, copy=None, odd=0, seed=0):
    """An optimiser over tensors that lie in one buffer, `odd` elements apart, with states as after
    some steps."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def lay(dtype, fill=None):
        flat = torch.full((sum(sizes) + odd * (len(sizes) + 1) + 16 * len(sizes) + 16,), 99, device="cuda").to(dtype)
        out, at = [], odd
        for n in sizes:
            out.append(flat[at:at + n])
            at = at + n + odd if odd else (at + n + 15) // 16 * 16
        for t in out:
            if fill is not None:
                t.copy_(fill(t.numel()))
        return flat, out

    def normal(scale):
        return lambda n: torch.randn(n, generator=g, device="cuda") * scale

    flat_p, params = lay(torch.float32, normal(0.05))
    _, grads = lay(grad_dtype, lambda n: torch.randn(n, generator=g, device="cuda") *
                   10 ** (torch.rand(n, generator=g, device="cuda") * 3 - 4))
    _, copies = lay(copy) if copy is not None else (None, None)
    m = [torch.randn(n, generator=g, device="cuda") * 10 ** (torch.rand(n, generator=g, device="cuda") * 3 - 4) for n in sizes]
    v = [t * t * (1 + torch.rand(len(t), generator=g, device="cuda")) for t in m]
    if bits == 32:
        flat_m, sm = lay(torch.float32)
        flat_v, sv = lay(torch.float32)
        states = {"m": sm, "v": sv}
        for a, b in ((sm, m), (sv, v)):
            for x, y in zip(a, b):
                x.copy_(y)
    else:
        flat_m, sm = lay(torch.int8)
        flat_v, sv = lay(torch.uint8)
        states = {"m": sm, "v": sv, "m_max": [], "v_max": []}
        for kind, held, given in (("m", sm, m), ("v", sv, v)):
            for x, y in zip(held, given):
                code, most = R.held(y.cpu().numpy(), kind, 4) if y.numel() else (np.zeros(0, np.int8), np.zeros(0, np.float32))
                x.copy_(torch.from_numpy(code))
                states[kind + "_max"].append(torch.from_numpy(most).cuda())
    opt = O.AdamW(params, grads, state_bits=bits, copies=copies, states=states, count=4)
    return opt, (flat_p, flat_m, flat_v)


def host(ts):
    return [t.detach().float().cpu().numpy().copy() for t in ts]


def read(opt):
    """What the optimiser holds, on the host; m and v as values (fp64) and, in 8 bits, as codes."""
    d = {"p": host(opt.params), "g": host(opt.grads)}
    if opt.state_bits == 32:
        return {**d, "m": host(opt.states["m"]), "v": host(opt.states["v"])}
    for k in ("m", "v"):
        d[k + "_code"] = [t.cpu().numpy().copy() for t in opt.states[k]]
        d[k + "_max"] = host(opt.states[k + "_max"])
        d[k] = [R.values(c, x, k) if len(c) else c for c, x in zip(d[k + "_code"], d[k + "_max"])]
    return d


def near(name, got, want, terms):
    assert got.shape == want.shape
    off = np.abs(got - want) - BOUND * terms
    assert got.size == 0 or off.max() <= 0, f"{name}: {off.max():.3e} over the bound"


def check_step(opt, before, after, step, clip=1.0, **kw):
    for k in range(len(opt.params)):
        if opt.params[k].numel() == 0:
            continue
        p, m, v = R.step64(before["p"][k], before["g"][k], before["m"][k], before["v"][k], step, clip=clip, **kw)
        # p is off by the rounding of its own size, of the update, and of an m' whose terms cancel
        # (they are at most about sqrt(v), so that part is off by 2^-24 lr or two)
        near(f"p[{k}]", after["p"][k], p, np.abs(before["p"][k]) + np.abs(p - before["p"][k]) * 4 + 1e-3)
        if opt.state_bits == 32:
            g = np.abs(before["g"][k]) * clip
            near(f"m[{k}]", after["m"][k], m, np.abs(before["m"][k]) + g)
            near(f"v[{k}]", after["v"][k], v, before["v"][k] + g * g)
        if opt.copies[k] is not None:
            want = torch.from_numpy(after["p"][k]).to(opt.copies[k].dtype)
            assert torch.equal(opt.copies[k].cpu(), want), f"copy[{k}]"


# ------------------------------------------------------------------------------ the format (CPU)

@pytest.mark.parametrize("kind,beta", [("m", 0.9), ("v", 0.999)])
def test_rounding_cancels_over_steps(kind, beta):
    """An average decays through 8 bits as it does without them: over 2000 steps of v -> 0.999 v (a
    seventh of one code's distance per step near the top, far less below) the mean of 4096 elements
    stays within a tenth, where rounding to the nearest code would leave it standing still."""
    x = np.linspace(0.3, 1.0, 4096).astype(np.float32)
    x[::R.BLOCK] = 1.0
    decay = np.float32(beta if kind == "v" else 0.999)
    code, most = R.held(x, kind, 0)
    for step in range(1, 2001):
        v = (R.values(code, most, kind).astype(np.float32) * decay).astype(np.float32)
        v[::R.BLOCK] = 1.0  # the block's maximum stays: nothing rescales the codes
        code, most = R.held(v, kind, step)
    rest = np.arange(4096) % R.BLOCK != 0
    want = x[rest].astype(np.float64).mean() * float(decay) ** 2000
    got = R.values(code, most, kind)[rest].mean()
    assert abs(got - want) < 0.1 * want, (got, want)


# ---------------------------------------------------------------------------------- refusals (CPU)

def tensors(n=4, **kw):
    t = (O.OptimTensor * 1)()
    fields = {**dict(param=256, grad=256, m=256, v=256, m_max=256, v_max=256, copy=None, n=n), **kw}
    for k, v in fields.items():
        setattr(t[0], k, v)
    return t


def adamw(t, count=1, clip=None, **kw):
    c = {**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, state_bits=32, grad_dtype=0,
                copy_dtype=1), **kw}
    return O._load().wtconv_adamw_step(count, t, O.AdamWConfig(**c), clip, None)


@pytest.mark.parametrize("kw,status", [
    (dict(lr=-1.0), W.ERR_INVALID_ARG), (dict(lr=float("nan")), W.ERR_INVALID_ARG), (dict(beta1=1.0), W.ERR_INVALID_ARG),
    (dict(beta2=-0.1), W.ERR_INVALID_ARG), (dict(eps=float("inf")), W.ERR_INVALID_ARG),
    (dict(weight_decay=-1.0), W.ERR_INVALID_ARG), (dict(step=0), W.ERR_INVALID_ARG),
    (dict(state_bits=16), W.ERR_UNSUPPORTED), (dict(grad_dtype=9), W.ERR_UNSUPPORTED), (dict(count=0), W.ERR_INVALID_ARG),
    (dict(clip=ctypes.c_void_p(258)), W.ERR_INVALID_ARG),
])
def test_step_refuses_scalars(kw, status):
    assert adamw(tensors(), **kw) == status


@pytest.mark.parametrize("kw,bits,status", [
    (dict(param=None), 32, W.ERR_INVALID_ARG), (dict(grad=None), 32, W.ERR_INVALID_ARG), (dict(m=None), 8, W.ERR_INVALID_ARG),
    (dict(v=258), 32, W.ERR_INVALID_ARG), (dict(m_max=None), 8, W.ERR_INVALID_ARG), (dict(v_max=257), 8, W.ERR_INVALID_ARG),
    (dict(copy=257), 32, W.ERR_INVALID_ARG), (dict(n=-1), 32, W.ERR_INVALID_ARG), (dict(n=1 << 41), 32, W.ERR_INVALID_ARG),
])
def test_step_refuses_tensors(kw, bits, status):
    assert adamw(tensors(**kw), state_bits=bits) == status


def test_norm_and_values_refuse(monkeypatch):
    lib, fake = O._load(), ctypes.c_void_p(256)
    assert adamw(tensors(copy=256), copy_dtype=0) == W.ERR_UNSUPPORTED
    assert adamw(None) == W.ERR_INVALID_ARG

    many = 10_000_000  # more elements than one launch sums: a workspace is needed

    def norm(t=tensors(n=many), dtype=0, most=1.0, out=fake, ws=fake, nbytes=1 << 16):
        return lib.wtconv_grad_norm(1, t, dtype, most, out, ws, nbytes, None)

    assert norm(out=None) == W.ERR_INVALID_ARG
    assert norm(most=0.0) == W.ERR_INVALID_ARG
    assert norm(most=float("nan")) == W.ERR_INVALID_ARG
    assert norm(dtype=4) == W.ERR_UNSUPPORTED
    assert norm(t=tensors(grad=None, n=many)) == W.ERR_INVALID_ARG
    assert lib.wtconv_grad_norm_workspace_size(1, tensors(n=many)) > 0
    assert lib.wtconv_grad_norm_workspace_size(1, tensors(n=-1)) == 0
    assert norm(ws=ctypes.c_void_p(264)) == W.ERR_INVALID_ARG
    assert norm(ws=None) == W.ERR_WORKSPACE
    assert norm(nbytes=7) == W.ERR_WORKSPACE
    assert lib.wtconv_adamw_state_values(1, tensors(), None, None, None) == W.ERR_INVALID_ARG
    one = (ctypes.c_void_p * 1)(None)
    assert lib.wtconv_adamw_state_values(1, tensors(), one, None, None) == W.ERR_INVALID_ARG
    monkeypatch.setenv("WTCONV_INJECT_FAULT", "1")
    assert norm() == W.ERR_INJECTED
    assert adamw(tensors()) == W.ERR_INJECTED


def test_binding_refuses():
    with pytest.raises(ValueError, match="no parameters"):
        O.AdamW([], [])
    with pytest.raises(ValueError, match="state_bits"):
        O.AdamW([torch.zeros(3)], [torch.zeros(3)], state_bits=4)
    with pytest.raises(ValueError, match=r"params\[0\]"):
        O.AdamW([torch.zeros(3)], [torch.zeros(3)])


# --------------------------------------------------------------------------------------- the kernels

@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("sizes", LISTS, ids=str)
@pytest.mark.parametrize("odd", [0, 3])
def test_step(sizes, grad, bits, odd):
    copy = None if grad == torch.float32 else (torch.bfloat16 if grad == torch.float16 else torch.float16)
    opt, flats = make(LISTS[sizes], grad, bits, copy, odd, seed=len(sizes))
    before = read(opt)
    gaps = [f.clone() for f in flats]
    opt.step()
    after = read(opt)
    check_step(opt, before, after, 5)
    if bits == 8:  # codes bit for bit, from the values that the codes before stand for in fp32
        for k, n in enumerate(LISTS[sizes]):
            if n == 0:
                continue
            m, v = (unit32(before[s + "_code"][k], before[s + "_max"][k], s) for s in "mv")
            m, v = R.averages32(before["g"][k], m, v)
            for name, x in (("m", m), ("v", v)):
                code, most = R.held(x, name, 5)
                assert np.array_equal(after[name + "_max"][k], most), (name, k)
                assert np.array_equal(after[name + "_code"][k], code), (name, k, np.sum(after[name + "_code"][k] != code))
    for flat, gap, ts in zip(flats, gaps, (opt.params, opt.states["m"], opt.states["v"])):  # nothing between them
        for t in ts:
            at = t.storage_offset()
            gap[at:at + t.numel()] = flat[at:at + t.numel()]
        assert torch.equal(gap, flat)


def unit32(code, most, kind):
    f = np.float32
    c = code.astype(f)
    unit = np.repeat(most * f(1.0 / R.TOP[kind] ** R.POWER[kind]), R.BLOCK)[:len(c)]
    return (c * np.abs(c)) * unit if kind == "m" else ((c * c) * (c * c)) * unit


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_steps(bits):
    opt, _ = make(LISTS["chunks"], torch.bfloat16, bits, torch.bfloat16, seed=3)
    before = read(opt)
    norm = float(np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in before["g"])))
    clip = opt.grad_norm(norm / 3)
    assert abs(float(clip[0]) - norm) < 1e-6 * norm and abs(float(clip[1]) - norm / 3 / (norm + 1e-6)) < 1e-6
    opt.step(clip=clip, lr=3e-4)
    check_step(opt, before, read(opt), 5, clip=float(clip[1]), lr=float(np.float32(3e-4)))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_many_steps_follow_fp64(bits):
    """Fifty steps from zero states on a quadratic: in 32 bits to fp32 rounding, in 8 bits to a few
    hundredths of the way that p went (a code is off by up to a sixteenth of its value, at random)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    target = torch.randn(3000, generator=g, device="cuda")
    p = torch.zeros(3000, device="cuda")
    grad = torch.zeros_like(p)
    opt = O.AdamW([p], [grad], state_bits=bits, lr=1e-2, weight_decay=0.1)
    p64, m64, v64, t64 = np.zeros(3000), np.zeros(3000), np.zeros(3000), target.double().cpu().numpy()
    for step in range(1, 51):
        torch.sub(p, target, out=grad)
        opt.step()
        p64, m64, v64 = R.step64(p64, p64 - t64, m64, v64, step, lr=1e-2, weight_decay=0.1)
    assert opt.count == 50
    off = np.abs(p.double().cpu().numpy() - p64)
    if bits == 32:
        assert off.max() < 1e-4 * np.abs(p64).max()
    else:
        assert off.mean() < 0.03 * np.abs(p64).mean()


@pytest.mark.gpu
@pytest.mark.parametrize("grad", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("sizes", LISTS, ids=str)
@pytest.mark.parametrize("odd", [0, 3])
def test_norm(sizes, grad, odd):
    opt, _ = make(LISTS[sizes], grad, 32, None, odd, seed=7)
    want = float(np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in host(opt.grads))))
    out = opt.grad_norm()
    assert abs(float(out[0]) - want) <= 1e-6 * want and float(out[1]) == 1.0
    again = opt.grad_norm(max_norm=want / 2)
    assert float(again[0]) == float(out[0]) and abs(float(again[1]) - want / 2 / (want + 1e-6)) < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("grad", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [7] * 20, [8, 31, 33, 255, 257, 1023, 1025, 2047, 2048, 2049, 4095], [2048 * 256],
                                   [2049] * 120, [1500] * 256, [1500] * 257], ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_of_few_chunks(sizes, grad, odd):
    """One launch (up to 256 chunks of 2048 elements) sums what 64 bits do, wherever chunks end.  A
    lane rounds 16 products and 2 sums before it moves to fp64, half of which reaches the root, and
    the root is rounded once."""
    g = torch.Generator().manual_seed(len(sizes))
    flat = [torch.randn(n + odd, generator=g).to(grad).cuda() for n in sizes]
    grads = [f[odd:] for f in flat]
    opt = O.AdamW([torch.zeros(n, device="cuda") for n in sizes], grads)
    want = float(np.sqrt(sum((t.double() ** 2).sum().item() for t in grads)))
    got = float(opt.grad_norm()[0])
    assert abs(got - want) <= (18 / 2 + 1) * 2.0**-24 * want
    for i in {0, len(sizes) // 2, len(sizes) - 1}:  # the last element counts
        grads[i][-1] = 1000.0
    want = float(np.sqrt(sum((t.double() ** 2).sum().item() for t in grads)))
    assert abs(float(opt.grad_norm()[0]) - want) <= (18 / 2 + 1) * 2.0**-24 * want


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e25])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_without_a_norm_changes_nothing(bad, bits):
    """Also where the squares overflow fp32 (1e25): the norm is infinite, the factor NaN."""
    opt, flats = make(LISTS["layer"], torch.float32, bits, seed=8)
    opt.grads[3][17] = bad
    before = [f.clone() for f in flats]
    clip = opt.grad_norm(1.0)
    assert not np.isfinite(float(clip[0])) and np.isnan(float(clip[1]))
    opt.step(clip=clip)
    for a, b in zip(before, flats):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_non_finite_gradients_without_clip():
    opt, _ = make([600], torch.float32, 32, seed=9)
    opt.grads[0][300] = float("nan")
    opt.step()
    for t in (opt.params[0], opt.states["m"][0], opt.states["v"][0]):
        bad = ~torch.isfinite(t)
        assert bad[300] and int(bad.sum()) == 1
    opt, _ = make([600], torch.float32, 8, seed=9)
    opt.grads[0][300] = float("nan")
    opt.step()
    m, v = opt.state_values()
    for t in (m[0], v[0]):  # its block, [256, 512), and nothing else
        assert torch.isnan(t[256:512]).all() and torch.isfinite(t[:256]).all() and torch.isfinite(t[512:]).all()
    assert int((~torch.isfinite(opt.params[0])).sum()) == 1


@pytest.mark.gpu
def test_zero_and_tiny_blocks():
    """Zero gradients on zero states, and averages below what a block can hold: no NaN, p only decays."""
    for bits in (32, 8):
        p = torch.ones(700, device="cuda")
        g = torch.zeros(700, device="cuda")
        g[300] = 1e-20
        opt = O.AdamW([p], [g], state_bits=bits, lr=0.1, weight_decay=0.5)
        opt.step()
        m, v = opt.state_values()
        assert torch.isfinite(m[0]).all() and torch.isfinite(v[0]).all()
        assert (m[0][:300] == 0).all() and float(v[0].max()) < 1e-42
        assert (p[:300] == p[0]).all() and abs(float(p[0]) - 0.95) < 1e-6


@pytest.mark.gpu
def test_state_values():
    opt, _ = make(LISTS["chunks"], torch.float32, 8, seed=10)
    held = read(opt)
    m, v = opt.state_values()
    for k in range(len(opt.params)):
        for got, name in ((m[k], "m"), (v[k], "v")):
            near(name, got.double().cpu().numpy(), held[name][k].astype(np.float64), np.abs(held[name][k]))
    opt32, _ = make([5], torch.float32, 32)
    assert opt32.state_values()[0][0] is opt32.states["m"][0]


@pytest.mark.gpu
def test_resume_graph_stream_and_new_gradients():
    """States adopted by a second optimiser, a captured step and another stream continue bit for bit."""
    runs = []
    for way in ("plain", "resume", "graph", "stream"):
        opt, flats = make(LISTS["layer"], torch.float32, 8, seed=11)
        opt.step()
        if way == "resume":
            d = opt.state_dict()
            opt = O.AdamW(opt.params, opt.grads, state_bits=8, states=d["states"], count=d["count"])
        opt.set_grads([g * 2 for g in opt.grads])
        torch.cuda.synchronize()
        if way == "graph":
            clip = opt.grad_norm(1.0)
            saved = [t.clone() for ts in (opt.params, *opt.states.values()) for t in ts]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.grad_norm(1.0, out=clip)
                opt.step(clip=clip)
            for t, s in zip([t for ts in (opt.params, *opt.states.values()) for t in ts], saved):
                t.copy_(s)
            graph.replay()
        elif way == "stream":
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                opt.step(clip=opt.grad_norm(1.0))
            side.synchronize()
        else:
            opt.step(clip=opt.grad_norm(1.0))
        torch.cuda.synchronize()
        assert opt.count == 6
        runs.append([t.clone() for ts in (opt.params, *opt.states.values()) for t in ts])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_elements_past_32_bits():
    """One tensor of more than 2^31 elements: its last block is updated like a small tensor's."""
    n = (1 << 31) + 700
    p = torch.empty(n, device="cuda")
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.empty(n, dtype=torch.int8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    blocks = -(-n // O.ADAMW_BLOCK)
    mm, vm = torch.ones(blocks, device="cuda"), torch.ones(blocks, device="cuda")
    tail = slice(n - 700, n)
    p.fill_(0.5), g.fill_(0), m.fill_(0), v.fill_(1)
    g[tail] = torch.linspace(-1, 1, 700, device="cuda")
    g0, p0 = g[tail].float().cpu().numpy(), p[tail].cpu().numpy()
    opt = O.AdamW([p], [g], state_bits=8, states={"m": [m], "v": [v], "m_max": [mm], "v_max": [vm]})
    clip = opt.grad_norm(1e9)
    want = float(np.sqrt((g0.astype(np.float64) ** 2).sum()))
    assert abs(float(clip[0]) - want) < 1e-6 * want
    opt.step()
    got, _, _ = R.step64(p0, g0, np.zeros(700), np.full(700, (1 / 255) ** 4), 1)
    near("p", p[tail].double().cpu().numpy(), got, np.abs(p0) * 4)
    assert float(m[tail].float().abs().max()) == 127 and int(m[: 1 << 20].abs().max()) == 0
    assert torch.equal(p[: 1 << 20], p[:1].expand(1 << 20))


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    p, g = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        O.AdamW([p], [g[:4]])
    with pytest.raises(ValueError, match="gradients"):
        O.AdamW([p], [g, g])
    with pytest.raises(ValueError, match=r"params\[0\]"):
        O.AdamW([p.half()], [g])
    with pytest.raises(ValueError, match="copies"):
        O.AdamW([p], [g], copies=[p])
    with pytest.raises(ValueError, match="states"):
        O.AdamW([p], [g], states={"m": [p]})
    with pytest.raises(ValueError, match=r"states\['m'\]"):
        O.AdamW([p], [g], state_bits=8, states={k: [p] for k in ("m", "v", "m_max", "v_max")})
    opt = O.AdamW([p, p.clone()], [g, g.clone()])
    before = bytes(opt._tensors)
    with pytest.raises(ValueError, match=r"grads\[1\]"):  # a refused list leaves the old one in place
        opt.set_grads([g.clone(), g[:4]])
    assert bytes(opt._tensors) == before
    with pytest.raises(W.WTConvError):
        opt.step(count=0)
    with pytest.raises(W.WTConvError):
        opt.step(lr=-1.0)
    assert opt.lr == 1e-3
    with pytest.raises(ValueError, match="clip"):
        opt.step(clip=torch.ones(1, device="cuda"))
    with pytest.raises(W.WTConvError):
        opt.grad_norm(-1.0)
    assert opt.count == 0
