"""The Int8 linear and its expert-grouped form, as measured cases.

Two operators, each with its input gradient:

- the linear with 8-bit weights and 8-bit tokens: every row of X (a token) and
  every row of W (an output channel) is held as int8 codes with one fp32 scale,
  Y = (codes_x codes_w^T) * scale_x * scale_w, and dX = dY W' with
  W' = bf16(codes_w * scale_w) for the frozen weight;
- the same products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of
  X belong to expert e, whose weight is W[e]; rows behind the last expert stay
  as they were.

With ``own`` false, ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the framework.
"""
import math

import torch

own = False

FWD, BWD, EFWD, EBWD = "linear_fwd", "linear_bwd", "expert_fwd", "expert_bwd"
_MAX_WORK = 2 * 8192 * 8192 * 8192  # operations of the largest listed case


def listed():
    return [
        # one token through a 13B attention projection: latency of the smallest call
        dict(name="fwd_1x5120x5120", op=FWD, M=1, N=5120, K=5120, quantized=False, out="bf16"),
        # a decode batch of 16 tokens through a 13B MLP projection: the weight stream
        dict(name="fwd_16x13824x5120", op=FWD, M=16, N=13824, K=5120, quantized=False, out="bf16"),
        # sizes that no tile divides, fp32 out (a small head over a short prompt)
        dict(name="fwd_333x1003x1111_fp32", op=FWD, M=333, N=1003, K=1111, quantized=False, out="fp32"),
        # 16 sequences of 256 tokens through a 7B MLP projection
        dict(name="fwd_4096x11008x4096", op=FWD, M=4096, N=11008, K=4096, quantized=False, out="bf16"),
        # a 65B projection whose tokens were quantized once for several projections
        dict(name="fwd_8192x8192x8192_quantized", op=FWD, M=8192, N=8192, K=8192, quantized=True, out="bf16"),
        # input gradients of a 13B projection on a short batch and of a 7B MLP projection on a full one
        dict(name="bwd_512x5120x5120", op=BWD, M=512, N=5120, K=5120),
        dict(name="bwd_4096x11008x4096", op=BWD, M=4096, N=11008, K=4096),
        # a decode batch spread over 8 wide experts: a few tokens each, the experts' weights stream
        dict(name="efwd_16_e8_11008x4096", op=EFWD, T=16, E=8, N=11008, K=4096, quantized=False, out="bf16", pad=0),
        # many narrow experts, ragged short row ranges (empty ones among them), rows behind the last expert
        dict(name="efwd_777_e60_1408x2048_pad", op=EFWD, T=777, E=60, N=1408, K=2048, quantized=False, out="bf16",
             pad=23),
        # a training batch over 16 experts
        dict(name="efwd_8192_e16_4096x2048", op=EFWD, T=8192, E=16, N=4096, K=2048, quantized=False, out="bf16",
             pad=0),
        # input gradients: short ragged ranges over many experts, and a training batch over wide ones
        dict(name="ebwd_1500_e64_1024x2048", op=EBWD, T=1500, E=64, N=1024, K=2048, pad=0),
        dict(name="ebwd_4096_e8_11008x4096", op=EBWD, T=4096, E=8, N=11008, K=4096, pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice((FWD, FWD, BWD, EFWD, EFWD, EBWD))
    while True:
        if op in (FWD, BWD):
            case = dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 22016), K=_log_int(rng, 64, 11008))
            rows, weights = case["M"], case["N"] * case["K"]
        else:
            case = dict(op=op, T=_log_int(rng, 1, 8192), E=_log_int(rng, 1, 128), N=_log_int(rng, 64, 11008),
                        K=_log_int(rng, 64, 4096), pad=rng.choice((0, rng.randint(1, 50))))
            rows, weights = case["T"], case["E"] * case["N"] * case["K"]
        if rng.random() < 0.5:  # aligned feature counts are the usual ones
            case["N"], case["K"] = -(-case["N"] // 64) * 64, -(-case["K"] // 64) * 64
        per_row = 2 * case["N"] * case["K"]
        if rows * per_row <= _MAX_WORK and weights <= (1 << 29):
            break
    if op in (FWD, EFWD):
        case["quantized"] = rng.random() < 0.3
        case["out"] = rng.choice(("bf16", "bf16", "fp32"))
    return case


# ---------------------------------------------------------------- inputs

def _quantize_rows(x):
    """Int8 codes and one fp32 scale for each row: c = RN32(127 / absmax),
    code = RN32(c x) rounded half away from zero, scale = RN32(absmax / 127).
    The quotients are taken in 64 bits and rounded once: torch divides by a
    number (and a number by a tensor) through a rounded reciprocal."""
    x = x.float()
    a = x.abs().amax(dim=-1, keepdim=True).double()
    c = torch.full_like(a, 127.0).div(a).float()
    c = torch.where(torch.isfinite(c), c, torch.zeros_like(c))
    v = (c * x).double()
    codes = torch.sign(v) * torch.floor(v.abs() + 0.5)
    scale = torch.where(c > 0, a.div(torch.full_like(a, 127.0)).float(), torch.zeros_like(c))
    return codes.to(torch.int8), scale.squeeze(-1)


def _offsets(T, E, gen):
    """Row ranges of a skewed router: E uneven shares of T rows, some empty."""
    share = torch.rand(E, generator=gen).pow(3) + 0.02
    pick = torch.multinomial(share, T, replacement=True, generator=gen)
    counts = torch.bincount(pick, minlength=E).tolist()
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return off


def _inputs(case, seed):
    """Activations, the frozen weight's codes and scales, and the row ranges."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    experts = case["op"] in (EFWD, EBWD)
    N, K = case["N"], case["K"]
    E = case["E"] if experts else 1
    rows = case["T"] + case["pad"] if experts else case["M"]
    codes = torch.empty((E, N, K), dtype=torch.int8, device=dev)
    scale = torch.empty((E, N), dtype=torch.float32, device=dev)
    for e in range(E):
        w = torch.randn((N, K), generator=g, device=dev) * 0.02
        w = torch.where(torch.rand((N, K), generator=g, device=dev) < 0.001, w * 8, w)
        codes[e], scale[e] = _quantize_rows(w)
    backward = case["op"] in (BWD, EBWD)
    width = N if backward else K
    act = torch.randn((rows, width), generator=g, device=dev)
    if backward:
        act = act * 0.01
    else:  # a few feature columns carry large values
        act[:, torch.randperm(width, generator=g, device=dev)[:max(1, width // 1000)]] *= 20
    out = {"act": act.to(torch.bfloat16), "codes": codes, "scale": scale, "offsets": [0, rows]}
    if experts:
        cpu = torch.Generator()
        cpu.manual_seed(seed + 1)
        out["offsets"] = _offsets(case["T"], E, cpu)
    return out


def _pad16(codes):
    """Rows of codes followed by zero codes up to a multiple of 16 bytes."""
    extra = -codes.shape[-1] % 16
    return torch.nn.functional.pad(codes, (0, extra)).contiguous()


def prepare(case, seed):
    """What the program holds: the activations (or the tokens it quantized
    before), the frozen weight, the experts' offsets, and for the expert
    products the buffer that receives the rows."""
    s = dict(case)
    d = _inputs(case, seed)
    experts = case["op"] in (EFWD, EBWD)
    if not experts:
        d["codes"], d["scale"] = d["codes"][0], d["scale"][0]
    s.update(d)
    N, K = case["N"], case["K"]
    dtype = torch.float32 if case.get("out") == "fp32" else torch.bfloat16
    s["dtype"] = dtype
    if experts:
        s["offsets_dev"] = torch.tensor(d["offsets"], dtype=torch.int32, device="cuda")
        width = N if case["op"] == EFWD else K
        s["buffer"] = torch.zeros((d["act"].shape[0], width), dtype=dtype, device="cuda")
    if case.get("quantized"):
        s["xcodes"], s["xscale"] = _quantize_rows(s.pop("act"))
    if own:
        import bit_nf4_quantized_13_b200 as q
        s["q"] = q
        shape = (case["E"], N, K) if experts else (N, K)
        s["w"] = q.Int8Rows(_pad16(s.pop("codes")), s.pop("scale"), shape)
        s["x"] = s["act"] if "act" in s else q.Int8Rows(_pad16(s.pop("xcodes")), s.pop("xscale"),
                                                        (d["act"].shape[0], K))
    return s


# ---------------------------------------------------------------- one pass

def _run_own(s):
    q, op = s["q"], s["op"]
    if op == FWD:
        return q.qlora_int8_linear_fwd(s["x"], s["w"], out_dtype=s["dtype"])
    if op == BWD:
        return q.qlora_int8_linear_bwd(s["x"], s["w"])
    if op == EFWD:
        return q.qlora_int8_expert_fwd(s["x"], s["w"], s["offsets_dev"], out_dtype=s["dtype"], Y=s["buffer"])
    return q.qlora_int8_expert_bwd(s["x"], s["w"], s["offsets_dev"], dX=s["buffer"])


def _forward_rows(xc, xs, wc, ws):
    return (xc.float() @ wc.float().t()) * xs[:, None] * ws[None, :]


def _backward_rows(dy, wc, ws):
    weight = (wc.float() * ws[:, None]).to(torch.bfloat16)
    return dy.float() @ weight.float()


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op in (BWD, EBWD):
        if op == BWD:
            return _backward_rows(s["act"], s["codes"], s["scale"]).to(torch.bfloat16)
        for e in range(s["E"]):
            lo, hi = s["offsets"][e], s["offsets"][e + 1]
            if hi > lo:
                s["buffer"][lo:hi] = _backward_rows(s["act"][lo:hi], s["codes"][e], s["scale"][e])
        return s["buffer"]
    xc, xs = (s["xcodes"], s["xscale"]) if "xcodes" in s else _quantize_rows(s["act"])
    if op == FWD:
        return _forward_rows(xc, xs, s["codes"], s["scale"]).to(s["dtype"])
    for e in range(s["E"]):
        lo, hi = s["offsets"][e], s["offsets"][e + 1]
        if hi > lo:
            s["buffer"][lo:hi] = _forward_rows(xc[lo:hi], xs[lo:hi], s["codes"][e], s["scale"][e])
    return s["buffer"]


def work(case):
    """Bytes and operations of one pass: activations in, the weights of the
    experts that a random router reaches, results out."""
    N, K = case["N"], case["K"]
    experts = case["op"] in (EFWD, EBWD)
    rows = case["T"] if experts else case["M"]
    hit = case["E"] * (1 - (1 - 1 / case["E"]) ** rows) if experts else 1
    weight = int(hit * (N * K + 4 * N))
    if case["op"] in (FWD, EFWD):
        x = rows * (K + 4) if case["quantized"] else 2 * rows * K
        y = rows * N * (4 if case["out"] == "fp32" else 2)
    else:
        x, y = 2 * rows * N, 2 * rows * K
    return {"bytes": x + weight + y, "flops": 2 * rows * N * K}


# ---------------------------------------------------------------- 64 bits

def _rows64(x):
    """The row quantization with each of its 32-bit steps taken as a 64-bit
    operation rounded once (exact products; quotients of 24-bit numbers round
    the same through 53 bits)."""
    x = x.double()
    top = x.abs().max(dim=1).values
    inv = (torch.full_like(top, 127.0) / top).float().double()
    live = torch.isfinite(inv)
    inv = inv.masked_fill(~live, 0.0)
    prod = (x * inv[:, None]).float().double()
    down = torch.trunc(prod)
    codes = down + torch.sign(prod) * ((prod - down).abs() >= 0.5)
    return codes, (top / torch.full_like(top, 127.0)).float().double().masked_fill(~live, 0.0)


def exact(case, seed):
    """The definition in 64 bits: integer sums are exact there."""
    d = _inputs(case, seed)
    off, act = d["offsets"], d["act"]
    backward = case["op"] in (BWD, EBWD)
    res = torch.zeros((act.shape[0], case["K"] if backward else case["N"]), dtype=torch.float64, device="cuda")
    if not backward:
        tokens, token_scale = _rows64(act)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if lo == hi:
            continue
        codes, scale = d["codes"][e].double(), d["scale"][e].double()
        if backward:
            held = (codes * scale.unsqueeze(1)).float().to(torch.bfloat16).double()  # the weight's compute type
            torch.mm(act[lo:hi].double(), held, out=res[lo:hi])
        else:
            sums = torch.einsum("mk,nk->mn", tokens[lo:hi], codes)
            res[lo:hi] = sums * torch.outer(token_scale[lo:hi], scale)
    return res
