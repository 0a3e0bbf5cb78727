"""The Int8 linear's definitions in 64 bits, for the tests: each 32-bit step
of the row quantization as a 64-bit operation rounded once, integer sums in
float64 (exact below 2^53), and the bounds of the kernels' own roundings."""
import torch

FLT_MAX = torch.finfo(torch.float32).max


def round32(t):
    return t.to(torch.float32).double()


def quantize_rows(x):
    """(codes float64, scale float64, bad rows) of the rows of x."""
    x = x.double()
    bad = ~torch.isfinite(x).all(dim=-1)
    a = x.abs().amax(dim=-1)
    a127 = torch.full_like(a, 127.0)
    c = round32(a127 / a)
    live = (a > 0) & (c <= FLT_MAX) & ~bad
    c = torch.where(live, c, torch.zeros_like(c))
    v = round32(torch.where(live[..., None], x, torch.zeros_like(x)) * c[..., None])
    codes = torch.sign(v) * torch.floor(v.abs() + 0.5)  # half away from zero (|v| < 2^7: the sum is exact)
    scale = torch.where(live, round32(a / a127), torch.zeros_like(a))
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return codes, scale, bad


def weight_rows(codes, scale, shape):
    """Codes (without their padding) and scales of an Int8Rows as float64."""
    return codes[..., :shape[-1]].double(), scale.double()


def forward(xc, xs, wc, ws):
    return (xc @ wc.transpose(-1, -2)) * xs[:, None] * ws[None, :]


def compute_weight(wc, ws):
    """W' = bf16(RN32(code * scale))."""
    return round32(wc * ws[:, None]).to(torch.bfloat16).double()


def check_forward(got, ref, name=""):
    """The sum is exact; its conversion to fp32 and the two products round
    once each (2^-24 relative), the result once to its own type; below the
    normal range a rounding is half the smallest subnormal instead."""
    eps = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    tiny = 2.0 ** -133 if got.dtype == torch.bfloat16 else 2.0 ** -148
    tol = ref.abs() * (eps + 3.01 * 2.0 ** -24 * (1 + eps)) + tiny
    _check(got, ref, tol, name)


def check_backward(got, dY, W, name=""):
    """Products of two bf16 values are exact in fp32.  N terms are added in
    some order: an addition that truncates is off by at most 2^-23 of the
    partial sum, and a partial sum is at most S = sum |dY W'| (1 + ...), so the
    sum is off by less than 1.01 N 2^-23 S (N <= 2^16); the result rounds once
    to bf16 (2^-8)."""
    ref = dY.double() @ W
    bound = dY.double().abs() @ W.abs()
    n = W.shape[0]
    tol = ref.abs() * 2.0 ** -8 + bound * (1.01 * n * 2.0 ** -23 * (1 + 2.0 ** -8)) + 2.0 ** -133
    _check(got, ref, tol, name)


def _check(got, ref, tol, name):
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()} against {ref[i].item()} (tolerance {tol[i].item():.3e})")


def check_differences(dX, dY, W, X, elements, h=0.5):
    """dX[m][k] for each (m, k) against a difference of the product: loss(X) =
    sum dY (X W^T) is linear in X, so (loss(X + h e) - loss(X - h e)) / 2 h is
    the derivative up to float64 roundings: two sums of M N terms, each a sum
    of K, off by less than (M N + K) 2^-52 of the sum of the terms' magnitudes.
    dX itself is off as check_backward derives, element by element."""
    dY64, n = dY.double(), W.shape[0]
    loss = lambda t: (dY64 * (t @ W.T)).sum().item()  # noqa: E731
    size = (dY64.abs() * ((X.abs() + h) @ W.abs().T)).sum().item()
    own = (dY.numel() + X.shape[1]) * 2.0 ** -52 * size / h
    bound = dY64.abs() @ W.abs()
    for m, k in elements:
        e = torch.zeros_like(X)
        e[m, k] = h
        d = (loss(X + e) - loss(X - e)) / (2 * h)
        tol = abs(d) * 2.0 ** -8 + bound[m, k].item() * (1.01 * n * 2.0 ** -23 * (1 + 2.0 ** -8)) + 1.01 * own
        got = dX[m, k].item()
        assert abs(got - d) <= tol, f"dX[{m}][{k}] = {got}, the product's difference {d} (tolerance {tol:.3e})"


def integer_gradient(generator, M, N, K, E=None):
    """(dY, codes, scale) of an exact gradient: dY integers up to 4, scales 1 or
    2 by channel, so W' = code * scale is exact in bf16 and every partial sum in
    any order is an integer below 2^24, exact in fp32 (N <= 16500)."""
    assert N * 127 * 2 * 4 < 2 ** 24
    lead = (N,) if E is None else (E, N)
    kw = dict(generator=generator, device=generator.device)
    codes = torch.randint(-127, 128, lead + (K,), dtype=torch.int8, **kw)
    scale = torch.randint(1, 3, lead, **kw).float()
    dY = torch.randint(-4, 5, (M, N), **kw).to(torch.bfloat16)
    return dY, codes, scale


def exact_gradient(dY, codes, scale):
    """bf16 of the exact sums: integers below 2^24, so float64 and fp32 hold them."""
    return (dY.double() @ (codes.double() * scale.double()[:, None])).float().to(torch.bfloat16)
