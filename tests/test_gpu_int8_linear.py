"""GPU parity of the Int8 linear (rows of Int8 codes, a scale per token and
output channel) and of its expert-grouped form against their definitions in
64 bits: codes, scales and untouched rows bit for bit, products within the
counted roundings.  Sizes from one row to several tiles, ragged row ranges,
masked (empty) experts, non-finite rows, streams and captured graphs."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import int8_reference as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import bit_nf4_quantized_13_b200 as q  # noqa: E402


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def tokens(seed, M, K, spread=1.0):
    x = torch.randn((M, K), generator=gen(seed), device="cuda") * spread
    x[:, K // 2] *= 8  # an outlier feature
    return x.to(torch.bfloat16)


def weight(seed, *shape):
    return q.qlora_int8_quantize_rows(torch.randn(shape, generator=gen(seed), device="cuda") * 0.02)


def fwd_ref(X, w, e=None):
    wc, ws = ref.weight_rows(w.codes, w.scale, w.shape)
    if e is not None:
        wc, ws = wc[e], ws[e]
    xc, xs, _ = ref.quantize_rows(X)
    return ref.forward(xc, xs, wc, ws)


def compute_weight(w, e=None):
    wc, ws = ref.weight_rows(w.codes, w.scale, w.shape)
    return ref.compute_weight(wc, ws) if e is None else ref.compute_weight(wc[e], ws[e])


# ----------------------------------------------------------------- quantizer

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 5120), (3, 15), (5, 16), (2, 17), (9, 1024), (8, 1025), (7, 2048),
                                    (1000, 333), (4, 2049), (3, 8192), (3, 8200), (2, 16385), (2, 40000),
                                    (257, 127), (333, 510), (65, 2047), (33, 4094), (33, 4099), (17, 8001),
                                    (4096, 512)])
def test_rows_match_the_definition(rows, K, dtype):
    x = (torch.randn((rows, K), generator=gen(rows + K), device="cuda") * 3).to(dtype)
    r = q.qlora_int8_quantize_rows(x)
    c, s, _ = ref.quantize_rows(x)
    assert torch.equal(r.codes[:, :K].double(), c)
    assert torch.equal(r.scale.double(), s)
    assert not r.codes[:, K:].any()  # the padding


def test_rows_zero_tiny_huge_and_ties():
    x = torch.zeros((9, 300), device="cuda")
    x[1, 5] = 1e-38          # c overflows: a zero row
    x[2, 7] = -4e-37         # just above: c = 127 / 4e-37 is finite
    x[3] = 3.0e38
    x[4] = -torch.finfo(torch.float32).max
    x[5, :3] = torch.tensor([127.0, 0.5, -1.5], device="cuda")  # halves go away from zero
    x[6] = 1e-45             # the smallest subnormal
    x[7, 299] = 2.0
    x[8] = -0.0
    r = q.qlora_int8_quantize_rows(x)
    c, s, _ = ref.quantize_rows(x)
    assert torch.equal(r.codes[:, :300].double(), c) and torch.equal(r.scale.double(), s)
    assert r.codes[5, :3].tolist() == [127, 1, -2]
    assert r.scale[0].item() == 0 and r.scale[1].item() == 0 and r.scale[6].item() == 0


@pytest.mark.parametrize("K", [40, 4096, 20001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_nonfinite_are_marked_alone(K, dtype):
    x = torch.randn((6, K), generator=gen(4), device="cuda").to(dtype)
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    q.qlora_int8_quantize_rows(x, status=st)
    assert st.item() == 0
    x[1, K - 1], x[3, 0], x[4, K // 2] = float("nan"), float("inf"), float("-inf")
    r = q.qlora_int8_quantize_rows(x, status=st)
    assert st.item() == 5
    c, s, bad = ref.quantize_rows(x)
    assert bad.tolist() == [False, True, False, True, True, False]
    assert torch.equal(r.scale.isnan(), bad)
    assert torch.equal(r.codes[:, :K].double(), c)  # codes 0 in the marked rows
    assert torch.equal(r.scale[~bad].double(), s[~bad])


# -------------------------------------------------------------- dense linear

FWD_SIZES = [(1, 1, 1), (1, 64, 64), (1, 5120, 512), (2, 33, 100), (3, 16, 4096), (7, 257, 1111), (8, 1000, 64),
             (9, 100, 5000), (15, 31, 48), (16, 512, 5120), (17, 130, 96), (31, 64, 1024), (33, 1003, 1111),
             (64, 300, 640), (100, 128, 3), (128, 256, 128), (130, 4097, 192), (255, 257, 129), (257, 512, 2048),
             (300, 1024, 8200), (512, 640, 384), (700, 333, 777), (1025, 1280, 4096), (2049, 2304, 1024), (300, 64, 11008), (40, 500, 9000),
             (257, 260, 8200)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", FWD_SIZES)
def test_linear_fwd(M, N, K, dtype):
    X, w = tokens(M + N, M, K), weight(K, N, K)
    Y = q.qlora_int8_linear_fwd(X, w, out_dtype=dtype)
    assert Y.dtype == dtype
    R = fwd_ref(X, w)
    ref.check_forward(Y, R, "Y")
    # tokens quantized before give the same bytes
    assert torch.equal(q.qlora_int8_linear_fwd(q.qlora_int8_quantize_rows(X), w, out_dtype=dtype), Y)
    assert q.qlora_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 64), (5, 100, 64), (16, 512, 1000), (33, 1003, 1111),
                                   (64, 8, 640), (100, 3, 128), (130, 4097, 192), (255, 129, 257), (300, 1024, 520),
                                   (512, 640, 384), (513, 72, 2049), (700, 333, 777), (1025, 1280, 2048),
                                   (2049, 2304, 1024), (256, 192, 9500), (257, 8, 96), (4608, 200, 4096),
                                   (4700, 68, 4100), (2600, 1, 8000), (1, 4096, 64), (40, 5000, 300), (300, 4100, 200),
                                   (257, 11008, 48)])
def test_linear_bwd(M, N, K):
    dY, w = tokens(M * 3 + N, M, N, 0.01), weight(K + 1, N, K)
    dX = q.qlora_int8_linear_bwd(dY, w)
    ref.check_backward(dX, dY, compute_weight(w), "dX")
    assert q.qlora_device_error() == 0


def test_largest_codes_fill_the_integer_sum():
    """K * 127^2 just below 2^31: the largest sums, positive and negative."""
    K = 131072
    w = q.qlora_int8_quantize_rows(torch.ones((70, K), device="cuda"))
    for M in (1, 40, 300):
        X = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
        X[M // 2] = -1
        Y = q.qlora_int8_linear_fwd(X, w, out_dtype=torch.float32)
        ref.check_forward(Y, fwd_ref(X, w), f"M = {M}")


@pytest.mark.parametrize("M", [4, 100, 600])
def test_nonfinite_and_zero_rows_stay_alone(M):
    N, K = 300, 640
    X, w = tokens(M, M, K), weight(3, N, K)
    clean = q.qlora_int8_linear_fwd(X, w)
    bad = X.clone()
    bad[1, 17], bad[M - 1, 0] = float("nan"), float("inf")
    bad[2] = 0
    Y = q.qlora_int8_linear_fwd(bad, w)
    assert Y[1].isnan().all() and Y[M - 1].isnan().all()
    assert not Y[2].any()
    keep = [m for m in range(M) if m not in (1, 2, M - 1)]
    assert torch.equal(Y[keep], clean[keep])
    # a NaN output channel, and a NaN row of dY
    w.scale[5] = float("nan")
    Y = q.qlora_int8_linear_fwd(X, w)
    assert Y[:, 5].isnan().all() and not Y[:, :5].isnan().any() and not Y[:, 6:].isnan().any()
    w.scale[5] = 0.01
    dY = tokens(7, M, N)
    clean = q.qlora_int8_linear_bwd(dY, w)
    dY[1, 3] = float("nan")
    dX = q.qlora_int8_linear_bwd(dY, w)
    assert dX[1].isnan().all()
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(dX[keep], clean[keep])


def test_small_and_large_scales_do_not_underflow_on_the_way():
    X = tokens(1, 40, 256) * 1e-30
    w = q.qlora_int8_quantize_rows(torch.randn((64, 256), generator=gen(2), device="cuda") * 1e25)
    ref.check_forward(q.qlora_int8_linear_fwd(X, w), fwd_ref(X, w))
    X = tokens(1, 40, 256) * 1e30
    w = q.qlora_int8_quantize_rows(torch.randn((64, 256), generator=gen(2), device="cuda") * 1e-30)
    ref.check_forward(q.qlora_int8_linear_fwd(X, w), fwd_ref(X, w))


def test_gradient_of_the_dequantized_product_by_differences():
    """The product with the dequantized weight is linear in X, so a difference
    quotient along any direction is <dX, direction> up to roundings: dX is off
    by at most 2^-8 relative per element plus the fp32 sum's error."""
    M, N, K = 40, 264, 320
    w, dY = weight(11, N, K), tokens(12, M, N, 0.1)
    W = compute_weight(w)
    dX = q.qlora_int8_linear_bwd(dY, w).double()
    X = torch.randn((M, K), generator=gen(13), device="cuda", dtype=torch.float64)
    for seed in range(4):
        D = torch.randn((M, K), generator=gen(20 + seed), device="cuda", dtype=torch.float64)
        loss = lambda t: (dY.double() * (t @ W.T)).sum()  # noqa: E731
        diff = (loss(X + 0.5 * D) - loss(X - 0.5 * D)).item()
        tol = (D.abs() * (dX.abs() * 1.01 * 2.0 ** -8 + 1.01 * N * 2.0 ** -23 * (dY.double().abs() @ W.abs()))).sum()
        # the quotient itself: two float64 sums of M N terms
        tol = tol.item() + 1e-9 * abs(loss(X).item()) + 1e-9
        assert abs(diff - (dX * D).sum().item()) <= tol


# --------------------------------------------------------------- by expert

def offsets_of(counts, first=0):
    off = [first]
    for n in counts:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


EXPERT_CASES = [
    # counts per expert, rows before, rows behind, N, K
    ([1], 0, 0, 64, 64),
    ([0], 0, 3, 100, 48),
    ([3, 0, 5], 0, 0, 130, 257),
    ([0, 0, 0, 2], 1, 2, 1003, 100),
    ([1, 1, 1, 1, 1, 1, 1, 1], 0, 0, 256, 1024),
    ([16, 17, 15, 1, 0, 33], 2, 9, 300, 333),
    ([2, 3, 0, 40, 1], 0, 7, 512, 2048),
    ([128, 64, 0, 1], 0, 0, 384, 128),
    ([100, 300, 0, 257, 5], 3, 23, 1408, 512),
    ([600, 0, 1, 511, 513], 0, 1, 520, 776),
    ([0] * 60 + [700] + [0] * 3, 0, 0, 72, 640),
    ([7] * 128, 0, 0, 96, 160),
    ([0, 1] * 500, 5, 5, 17, 33),
    ([3900, 100, 0, 150], 1, 3, 72, 300),   # many full tiles, small ones among them
    ([1500, 2600, 1025], 0, 0, 65, 513),
    ([5, 0, 30], 2, 1, 5000, 130),          # few tiles, a long contraction of the gradient
    ([300, 20], 0, 4, 4097, 64),
    ([18, 0, 30], 1, 2, 100, 8300),         # and of the forward
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,before,behind,N,K", EXPERT_CASES)
def test_expert_fwd(counts, before, behind, N, K, dtype):
    E, T = len(counts), sum(counts) + before + behind
    off = offsets_of(counts, before)
    X, w = tokens(N + T, T, K), weight(K, E, N, K)
    Y = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    assert q.qlora_int8_expert_fwd(X, w, off, Y=Y) is Y
    o = off.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            ref.check_forward(Y[o[e]:o[e + 1]], fwd_ref(X[o[e]:o[e + 1]], w, e), f"expert {e}")
    assert (Y[:o[0]] == 7).all() and (Y[o[-1]:] == 7).all()
    Y2 = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    q.qlora_int8_expert_fwd(q.qlora_int8_quantize_rows(X), w, off, Y=Y2)
    assert torch.equal(Y, Y2)
    assert q.qlora_device_error() == 0


@pytest.mark.parametrize("counts,before,behind,N,K", EXPERT_CASES)
def test_expert_bwd(counts, before, behind, N, K):
    E, T = len(counts), sum(counts) + before + behind
    off = offsets_of(counts, before)
    dY, w = tokens(N + T + 1, T, N, 0.01), weight(K + 2, E, N, K)
    dX = torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    assert q.qlora_int8_expert_bwd(dY, w, off, dX=dX) is dX
    o = off.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            ref.check_backward(dX[o[e]:o[e + 1]], dY[o[e]:o[e + 1]], compute_weight(w, e), f"expert {e}")
    assert (dX[:o[0]] == 7).all() and (dX[o[-1]:] == 7).all()
    assert q.qlora_device_error() == 0


def test_experts_equal_the_dense_linear():
    """Each expert's rows are exactly the dense call's on those rows: the
    forward's sums are exact, so the bytes agree whatever kernel ran."""
    counts, N, K = [40, 0, 3, 300], 640, 512
    off = offsets_of(counts)
    X, w = tokens(5, sum(counts), K), weight(6, len(counts), N, K)
    Y = q.qlora_int8_expert_fwd(X, w, off)
    o = off.tolist()
    for e in range(len(counts)):
        if counts[e]:
            we = q.Int8Rows(w.codes[e].contiguous(), w.scale[e].contiguous(), (N, K))
            assert torch.equal(Y[o[e]:o[e + 1]], q.qlora_int8_linear_fwd(X[o[e]:o[e + 1]].contiguous(), we))


@pytest.mark.parametrize("off", [[0, 10 ** 6, 2 * 10 ** 6], [-5, 20, 10 ** 9], [30, 10, 50], [2 ** 31 - 1, -2 ** 31, 0]])
def test_offsets_outside_the_rows_are_clamped(off):
    """Offsets that no router writes stay inside the T rows: the guard rows on
    both sides of the outputs keep their bytes."""
    T, N, K = 50, 96, 64
    w = weight(1, 2, N, K)
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for width, call in ((N, lambda t, o: q.qlora_int8_expert_fwd(t, w, offsets, Y=o)),
                        (K, lambda t, o: q.qlora_int8_expert_bwd(t, w, offsets, dX=o))):
        big = torch.full((3 * T, width), 7.0, dtype=torch.bfloat16, device="cuda")
        call(tokens(2, T, K if width == N else N), big[T:2 * T])
        torch.cuda.synchronize()
        assert (big[:T] == 7).all() and (big[2 * T:] == 7).all()
    assert q.qlora_device_error() == 0


# ------------------------------------------------- streams, graphs, together

def test_empty_batches():
    w = weight(1, 64, 48)
    X = torch.empty((0, 48), dtype=torch.bfloat16, device="cuda")
    assert q.qlora_int8_linear_fwd(X, w).shape == (0, 64)
    assert q.qlora_int8_linear_bwd(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 48)
    r = q.qlora_int8_quantize_rows(X)
    assert r.codes.shape == (0, 48) and r.scale.shape == (0,)
    we = weight(1, 2, 64, 48)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert q.qlora_int8_expert_fwd(X, we, off).shape == (0, 64)


@pytest.mark.parametrize("M", [1, 16, 40, 500])
def test_calls_on_another_stream(M):
    N, K = 700, 1024
    X, w, dY = tokens(M, M, K), weight(2, N, K), tokens(M + 1, M, N)
    Y0, dX0 = q.qlora_int8_linear_fwd(X, w), q.qlora_int8_linear_bwd(dY, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [(q.qlora_int8_linear_fwd(X, w, stream=side), q.qlora_int8_linear_bwd(dY, w, stream=side))
            for _ in range(8)]
    with torch.cuda.stream(side):
        outs.append((q.qlora_int8_linear_fwd(X, w), q.qlora_int8_linear_bwd(dY, w)))
    torch.cuda.current_stream().wait_stream(side)
    for Y, dX in outs:
        assert torch.equal(Y, Y0) and torch.equal(dX, dX0)


@pytest.mark.parametrize("T", [12, 300, 1500])
def test_graph_replays_follow_inputs_and_offsets(T):
    E, N, K = 6, 520, 640
    w = weight(3, E, N, K)
    X, dY = tokens(1, T, K), tokens(2, T, N, 0.01)
    off = offsets_of([T // 2, 0, T - T // 2, 0, 0, 0])
    Y, dX = q.qlora_int8_expert_fwd(X, w, off), q.qlora_int8_expert_bwd(dY, w, off)  # first calls outside capture
    Yd = q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes[0], w.scale[0], (N, K)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_int8_expert_fwd(X, w, off, Y=Y)
        q.qlora_int8_expert_bwd(dY, w, off, dX=dX)
        q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes[0], w.scale[0], (N, K)), Y=Yd)
    for seed, counts in ((5, [0, T, 0, 0, 0, 0]), (6, [T // 6, T // 3, 0, 1, T - T // 6 - T // 3 - 1, 0])):
        X.copy_(tokens(seed, T, K))
        dY.copy_(tokens(seed + 10, T, N, 0.01))
        off.copy_(offsets_of(counts))
        for _ in range(2):
            graph.replay()
        o = off.tolist()
        for e in range(E):
            if counts[e]:
                ref.check_forward(Y[o[e]:o[e + 1]], fwd_ref(X[o[e]:o[e + 1]], w, e), f"expert {e}")
                ref.check_backward(dX[o[e]:o[e + 1]], dY[o[e]:o[e + 1]], compute_weight(w, e), f"expert {e}")
        ref.check_forward(Yd, fwd_ref(X, w, 0), "dense")


def test_an_expert_block_forward_and_back():
    """Router order, gate and up on tokens quantized once, down, and the input
    gradients of all three: each call against the definition on its own
    inputs, rows of no expert untouched."""
    T, E, H, F = 333, 5, 512, 776
    g = gen(9)
    choice = torch.randint(0, E + 1, (T,), generator=g, device="cuda")  # expert E: dropped tokens
    order = torch.argsort(choice, stable=True)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(choice, minlength=E + 1)[:E].cumsum(0).to(torch.int32)
    o = off.tolist()
    X = tokens(10, T, H)[order].contiguous()
    gate, up, down = weight(1, E, F, H), weight(2, E, F, H), weight(3, E, H, F)
    xq = q.qlora_int8_quantize_rows(X)
    zeros = lambda n: torch.zeros((T, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    G, U = q.qlora_int8_expert_fwd(xq, gate, off, Y=zeros(F)), q.qlora_int8_expert_fwd(xq, up, off, Y=zeros(F))
    A = (torch.nn.functional.silu(G.float()) * U.float()).to(torch.bfloat16)
    Y = q.qlora_int8_expert_fwd(A, down, off, Y=zeros(H))
    dY = tokens(12, T, H, 0.01)
    dA = q.qlora_int8_expert_bwd(dY, down, off, dX=zeros(F))
    sig = torch.sigmoid(G.float())
    dU = (dA.float() * G.float() * sig).to(torch.bfloat16)
    dG = (dA.float() * U.float() * sig * (1 + G.float() * (1 - sig))).to(torch.bfloat16)
    dX = q.qlora_int8_expert_bwd(dG, gate, off, dX=zeros(H)), q.qlora_int8_expert_bwd(dU, up, off, dX=zeros(H))
    for e in range(E):
        s = slice(o[e], o[e + 1])
        for got, x, w in ((G, X, gate), (U, X, up), (Y, A, down)):
            ref.check_forward(got[s], fwd_ref(x[s], w, e), f"expert {e}")
        for got, d, w in ((dA, dY, down), (dX[0], dG, gate), (dX[1], dU, up)):
            ref.check_backward(got[s], d[s], compute_weight(w, e), f"expert {e}")
    for t in (G, U, Y, dA, *dX):
        assert not t[o[-1]:].any()


@pytest.mark.parametrize("M,N,K", [(200, 4100, 1024), (300, 5120, 640), (400, 2560, 6200), (512, 4608, 300),
                                   (777, 5000, 512), (1500, 5120, 256), (512, 2049, 7000), (200, 5000, 9000)])
def test_linear_fwd_between_the_tile_widths(M, N, K):
    """Batches of a few tiles, whose width follows the number of SM pairs."""
    X, w = tokens(M + N, M, K), weight(K, N, K)
    ref.check_forward(q.qlora_int8_linear_fwd(X, w), fwd_ref(X, w), "Y")
    assert q.qlora_device_error() == 0


def test_two_streams_at_once():
    """Independent calls on two streams, each with its own buffers."""
    T, E, N, K = 700, 4, 1100, 2048
    w = weight(3, E, N, K)
    X, dY = tokens(1, T, K), tokens(2, T, N, 0.01)
    off = offsets_of([100, 0, 350, 200], 7)
    full = lambda n: torch.full((T, n), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Y0, dX0 = q.qlora_int8_expert_fwd(X, w, off, Y=full(N)), q.qlora_int8_expert_bwd(dY, w, off, dX=full(K))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    bufs = [[(full(N), full(K)) for _ in range(10)] for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(10):
        for s, b in zip(streams, bufs):
            outs.append((q.qlora_int8_expert_fwd(X, w, off, Y=b[i][0], stream=s),
                         q.qlora_int8_expert_bwd(dY, w, off, dX=b[i][1], stream=s)))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for Y, dX in outs:
        assert torch.equal(Y, Y0) and torch.equal(dX, dX0)
    assert q.qlora_device_error() == 0


def test_two_graphs_on_one_workspace():
    """Graphs replayed in turn on one stream may share a workspace."""
    M, N, K = 500, 512, 11008
    w, shapes = weight(4, N, K), ((500, 1), (300, 2))
    need = max(max(q.qlora_int8_linear_fwd_workspace_size(m, N, K), q.qlora_int8_linear_bwd_workspace_size(m, N, K))
               for m, _ in shapes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    runs = []
    for m, seed in shapes:
        X, dY = tokens(seed, m, K), tokens(seed + 5, m, N, 0.01)
        want = q.qlora_int8_linear_fwd(X, w), q.qlora_int8_linear_bwd(dY, w)
        got = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.qlora_int8_linear_fwd(X, w, Y=got[0], ws=ws)
            q.qlora_int8_linear_bwd(dY, w, dX=got[1], ws=ws)
        runs.append((graph, X, dY, want, got))
    ws.fill_(255)
    for _ in range(3):
        for graph, _, _, _, got in runs:
            for t in got:
                t.fill_(float("nan"))
            graph.replay()
        for _, _, _, want, got in runs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def check_ends(M, a, b, check):
    for s in (slice(0, 3), slice(M - 70, M)):
        check(a[s], b[s])


def test_offsets_past_32_bits():
    """Tokens, outputs and gradients of more than 2^31 elements, and weights of
    more than 2^31 codes: the last rows are as right as the first."""
    M, big, few = (1 << 20) + 77, 2064, 24
    X, w = tokens(1, M, few), weight(2, big, few)
    Y = q.qlora_int8_linear_fwd(X, w)
    check_ends(M, X, Y, lambda x, y: ref.check_forward(y, fwd_ref(x, w), "wide output"))
    del Y
    w = weight(3, few, big)
    dX = q.qlora_int8_linear_bwd(X, w)
    check_ends(M, X, dX, lambda d, x: ref.check_backward(x, d, compute_weight(w), "gradient"))
    Y = q.qlora_int8_linear_fwd(dX, w)
    check_ends(M, dX, Y, lambda x, y: ref.check_forward(y, fwd_ref(x, w), "long input"))
    del dX, Y, X
    E, N, K = 66, 8000, 4112
    w = q.alloc_int8_rows((E, N, K), "cuda")
    for e in range(E):
        q.qlora_int8_quantize_rows(torch.randn((N, K), generator=gen(e), device="cuda") * 0.02,
                                   out=q.Int8Rows(w.codes[e], w.scale[e], (N, K)))
    for counts in ([3] + [0] * 64 + [4], [30] + [0] * 64 + [100]):
        off, T = offsets_of(counts), sum(counts)
        X, dY = tokens(T, T, K), tokens(T + 1, T, N, 0.01)
        Y, dX = q.qlora_int8_expert_fwd(X, w, off), q.qlora_int8_expert_bwd(dY, w, off)
        for e, s in ((0, slice(0, counts[0])), (E - 1, slice(counts[0], T))):
            we = q.Int8Rows(w.codes[e], w.scale[e], (N, K))
            ref.check_forward(Y[s], fwd_ref(X[s], we), f"expert {e}")
            ref.check_backward(dX[s], dY[s], compute_weight(we), f"expert {e}")
    assert q.qlora_device_error() == 0


def test_threads_on_their_own_streams():
    N, K, sizes = 300, 640, (400, 2, 64, 200)
    X, dY, w = tokens(1, 400, K), tokens(2, 400, N, 0.01), weight(3, N, K)
    want = {m: (q.qlora_int8_linear_fwd(X[:m], w), q.qlora_int8_linear_bwd(dY[:m], w)) for m in sizes}
    torch.cuda.synchronize()
    got = {}

    def run(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            outs = []
            for i in range(40):
                m = sizes[(i + k) % 4]
                outs.append((m, q.qlora_int8_linear_fwd(X[:m], w), q.qlora_int8_linear_bwd(dY[:m], w)))
            stream.synchronize()
        got[k] = outs

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(got) == [0, 1, 2, 3]
    for outs in got.values():
        for m, Y, dX in outs:
            assert torch.equal(Y, want[m][0]) and torch.equal(dX, want[m][1])


FIRST_CALLS_CAPTURED = """
import torch, bit_nf4_quantized_13_b200 as q
w = q.qlora_int8_quantize_rows(torch.randn(2, 300, 640, device="cuda"))
X = torch.randn(400, 640, device="cuda").bfloat16()
dY = torch.randn(400, 300, device="cuda").bfloat16()
off = torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
def calls():
    return (q.qlora_int8_expert_fwd(X, w, off), q.qlora_int8_expert_fwd(X[:3], w, off), q.qlora_int8_expert_fwd(X[:12], w, off),
            q.qlora_int8_expert_bwd(dY, w, off), q.qlora_int8_quantize_rows(X).codes)
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
assert q.qlora_device_error() == 0
"""


def test_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------ outputs that the call makes

def poison(shape, dtype, copies=4):
    """Leaves freed blocks of this size behind that hold NaN, for the allocator to hand out again."""
    blocks = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(copies)]
    torch.cuda.synchronize()
    del blocks


def check_zeros_outside(out, off, check):
    """Expert e's rows hold what check(e, rows) says, every other row zeros."""
    o = off.tolist()
    for e in range(len(o) - 1):
        if o[e + 1] > o[e]:
            check(e, slice(o[e], o[e + 1]))
    assert not out[:o[0]].any() and not out[o[-1]:].any()


MADE_CASES = [
    # counts per expert, rows before, rows behind, N, K
    ([0, 1], 1, 1, 33, 17),
    ([3, 0, 4], 2, 3, 64, 48),
    ([0, 0], 0, 40, 97, 130),          # no expert has rows
    ([1, 2, 0, 5], 3, 2, 130, 257),
    ([20, 0, 13], 5, 12, 96, 64),
    ([700, 0, 300, 2], 100, 398, 131, 520),
    ([50, 14], 0, 0, 65, 33),          # every row belongs to one
]


@pytest.mark.parametrize("counts,before,behind,N,K", MADE_CASES)
def test_outputs_made_by_an_expert_call_hold_zeros_where_no_expert_has_rows(counts, before, behind, N, K):
    E, T = len(counts), sum(counts) + before + behind
    off = offsets_of(counts, before)
    X, dY, w = tokens(1, T, K), tokens(2, T, N, 0.01), weight(3, E, N, K)
    xq = q.qlora_int8_quantize_rows(X)
    side = torch.cuda.Stream()
    for dtype in (torch.bfloat16, torch.float32):
        for x in (X, xq):
            for stream in (None, side):
                poison((T, N), dtype)
                Y = q.qlora_int8_expert_fwd(x, w, off, out_dtype=dtype, stream=stream)
                torch.cuda.synchronize()
                check_zeros_outside(Y, off, lambda e, s: ref.check_forward(Y[s], fwd_ref(X[s], w, e), f"expert {e}"))
    poison((T, K), torch.bfloat16)
    dX = q.qlora_int8_expert_bwd(dY, w, off)
    check_zeros_outside(dX, off, lambda e, s: ref.check_backward(dX[s], dY[s], compute_weight(w, e), f"expert {e}"))
    assert q.qlora_device_error() == 0


@pytest.mark.parametrize("T", [6, 40, 600])
def test_a_graph_clears_the_rows_that_lose_their_expert(T):
    """Outputs made inside a capture: rows that had an expert in the last replay and have none in this one are zeros."""
    N, K = 72, 136
    w = weight(3, 2, N, K)
    X, dY = tokens(1, T, K), tokens(2, T, N, 0.01)
    off = offsets_of([T // 2, T - T // 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, dX = q.qlora_int8_expert_fwd(X, w, off), q.qlora_int8_expert_bwd(dY, w, off)
    for counts, first in (([T // 2, T - T // 2], 0), ([1, T // 3], T // 3), ([0, 0], T), ([T - 1, 0], 1)):
        off.copy_(offsets_of(counts, first))
        graph.replay()
        check_zeros_outside(Y, off, lambda e, s: ref.check_forward(Y[s], fwd_ref(X[s], w, e), f"expert {e}"))
        check_zeros_outside(dX, off,
                            lambda e, s: ref.check_backward(dX[s], dY[s], compute_weight(w, e), f"expert {e}"))


def test_zeroed_rows_past_32_bits():
    T, N, K = (1 << 20) + 77, 2064, 24
    X, w = tokens(1, T, K), weight(2, 2, N, K)
    off = offsets_of([3, 40], T - 60)
    poison((T, N), torch.bfloat16, copies=1)
    Y = q.qlora_int8_expert_fwd(X, w, off)
    check_zeros_outside(Y, off, lambda e, s: ref.check_forward(Y[s], fwd_ref(X[s], w, e), f"expert {e}"))


# ------------------------------------------------------- offsets out of order

def in_order(off, T):
    """How offsets are read: clamped to [0, T], each no less than the one before it."""
    out = [min(max(off[0], 0), T)]
    for o in off[1:]:
        out.append(max(out[-1], min(o, T)))
    return out


SCRAMBLED = [[5, 2, 8], [0, 8, 3, 8], [-5, 2, 10 ** 9], [30, 10, 50], [2 ** 31 - 1, -2 ** 31, 0], [0, 10 ** 6, 2, 10 ** 6],
             [1, 1, 0, 2, 1, 3, 0, 2], [4 * (i % 5) - i % 7 for i in range(71)], [2 - i % 3 for i in range(1025)]]


@pytest.mark.parametrize("off", SCRAMBLED, ids=lambda o: f"{len(o) - 1}_experts_from_{o[0]}_{o[1]}")
@pytest.mark.parametrize("T", [1, 3, 8, 12, 50, 300])
def test_offsets_out_of_order_mean_the_same_for_every_batch(T, off):
    """Whichever kernel a batch of this size takes."""
    E, N, K = len(off) - 1, 96, 64
    w = weight(1, E, N, K)
    X, dY = tokens(2, T, K), tokens(3, T, N, 0.01)
    offsets, o = torch.tensor(off, dtype=torch.int32, device="cuda"), in_order(off, T)
    full = lambda n: torch.full((T, n), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    Y, Yq = full(N), full(N)
    q.qlora_int8_expert_fwd(X, w, offsets, Y=Y)
    q.qlora_int8_expert_fwd(q.qlora_int8_quantize_rows(X), w, offsets, Y=Yq)
    dX = q.qlora_int8_expert_bwd(dY, w, offsets, dX=full(K))
    for e in range(E):
        s = slice(o[e], o[e + 1])
        if o[e + 1] > o[e]:
            ref.check_forward(Y[s], fwd_ref(X[s], w, e), f"expert {e}")
            ref.check_backward(dX[s], dY[s], compute_weight(w, e), f"expert {e}")
    for t in (Y, dX):
        assert (t[:o[0]] == 7).all() and (t[o[-1]:] == 7).all()
    assert torch.equal(Y, Yq)
    assert q.qlora_device_error() == 0


# ------------------------------------------- the gradient, element by element

def test_gradient_elements_by_differences():
    """Single elements of dX against differences of the product along their own
    direction (a sum over all elements would hide a wrong one)."""
    M, N, K = 40, 264, 320
    w, dY = weight(11, N, K), tokens(12, M, N, 0.1)
    dX = q.qlora_int8_linear_bwd(dY, w)
    X = torch.randn((M, K), generator=gen(13), device="cuda", dtype=torch.float64)
    picks = torch.stack([torch.randint(0, n, (120,), generator=gen(14), device="cuda") for n in (M, K)], 1).tolist()
    ref.check_differences(dX, dY, compute_weight(w), X, picks + [[m, k] for m in (0, M - 1) for k in (0, K - 1)])


def int8_rows(codes, scale):
    shape = tuple(codes.shape)
    return q.Int8Rows(torch.nn.functional.pad(codes, (0, -shape[-1] % 16)).contiguous(), scale, shape)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (16, 63, 40), (3, 65, 130), (40, 4097, 200), (100, 8192, 64),
                                   (257, 11008, 48), (16, 11008, 512), (16, 5120, 5120), (513, 4160, 300),
                                   (500, 10000, 128), (1, 16500, 1000), (300, 16385, 33), (600, 8200, 776),
                                   (2049, 2304, 1024), (4700, 4100, 68)])
def test_gradient_of_integers_is_exact(M, N, K):
    """Every term counts, whole tiles and parts: nothing rounds before the result."""
    dY, codes, scale = ref.integer_gradient(gen(M + N), M, N, K)
    assert torch.equal(q.qlora_int8_linear_bwd(dY, int8_rows(codes, scale)), ref.exact_gradient(dY, codes, scale))
    assert q.qlora_device_error() == 0


@pytest.mark.parametrize("counts,before,behind,N,K", [([5, 0, 30], 2, 1, 5000, 130), ([300, 20], 0, 4, 4097, 64),
                                                      ([70], 3, 5, 8192, 64), ([600, 0, 1, 511, 513], 0, 1, 4160, 776),
                                                      ([1] * 40, 0, 0, 2049, 100), ([16, 2, 0, 33], 1, 0, 11008, 300),
                                                      ([3900, 100, 0, 150], 1, 3, 72, 300)])
def test_expert_gradient_of_integers_is_exact(counts, before, behind, N, K):
    E, T = len(counts), sum(counts) + before + behind
    off = offsets_of(counts, before)
    dY, codes, scale = ref.integer_gradient(gen(T + N), T, N, K, E)
    dX = torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    q.qlora_int8_expert_bwd(dY, int8_rows(codes, scale), off, dX=dX)
    o = off.tolist()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        assert torch.equal(dX[s], ref.exact_gradient(dY[s], codes[e], scale[e])), f"expert {e}"
    assert (dX[:o[0]] == 7).all() and (dX[o[-1]:] == 7).all()


@pytest.mark.parametrize("N,K", [(65, 300), (264, 5120), (4097, 200), (8192, 64), (11008, 48)])
def test_gradient_of_one_channel_is_its_weight(N, K):
    """dY = one 1 a row: dX is that channel's W' = bf16(RN32(code * scale)),
    rounded and not truncated, bit for bit.  All channels at once, and a few
    rows whose tiles are cut along the contraction."""
    w = weight(N + K, N, K)
    W = compute_weight(w).to(torch.bfloat16)
    assert torch.equal(q.qlora_int8_linear_bwd(torch.eye(N, dtype=torch.bfloat16, device="cuda"), w), W)
    edges = [n for b in range(64, N, 64) for n in (b - 1, b)] + [0, N - 1]
    for first in range(0, len(edges), 100):
        at = torch.tensor(edges[first:first + 100], device="cuda")
        dY = torch.zeros((len(at), N), dtype=torch.bfloat16, device="cuda")
        dY[torch.arange(len(at), device="cuda"), at] = 1
        assert torch.equal(q.qlora_int8_linear_bwd(dY, w), W[at])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(9, 9217, 130), (12, 9472, 1111), (16, 13824, 5120), (13, 20001, 64), (16, 9216, 300)])
def test_linear_fwd_of_a_decode_batch_over_a_wide_weight(M, N, K, dtype):
    """9 to 16 tokens on both sides of the width from which the tensor-core
    kernel's tiles fill half of the SM pairs (more than 36 tiles of 256 channels)."""
    X, w = tokens(M + N, M, K), weight(K, N, K)
    Y = q.qlora_int8_linear_fwd(X, w, out_dtype=dtype)
    ref.check_forward(Y, fwd_ref(X, w), "Y")
    assert torch.equal(q.qlora_int8_linear_fwd(q.qlora_int8_quantize_rows(X), w, out_dtype=dtype), Y)
    assert q.qlora_device_error() == 0


@pytest.mark.parametrize("counts,before,behind,N,K", [([70], 3, 5, 64, 11008), ([300], 0, 212, 130, 9000), ([1], 511, 0, 512, 4096),
                                                      ([0], 9, 0, 64, 11008), ([2], 3, 1, 700, 4096)])
def test_one_expert_that_has_some_of_the_rows(counts, before, behind, N, K):
    """What the host cuts for all T rows, the device cuts for the expert's."""
    T, off = sum(counts) + before + behind, offsets_of(counts, before)
    s = slice(before, before + counts[0])
    X, dY, w = tokens(T, T, K), tokens(T + 1, T, N, 0.01), weight(K, 1, N, K)
    Y, dX = q.qlora_int8_expert_fwd(X, w, off), q.qlora_int8_expert_bwd(dY, w, off)
    check_zeros_outside(Y, off, lambda e, s: ref.check_forward(Y[s], fwd_ref(X[s], w, e)))
    check_zeros_outside(dX, off, lambda e, s: ref.check_backward(dX[s], dY[s], compute_weight(w, e)))
    dense = q.Int8Rows(w.codes[0], w.scale[0], (N, K))
    if counts[0]:
        assert torch.equal(Y[s], q.qlora_int8_linear_fwd(X[s].clone(), dense))
    assert q.qlora_device_error() == 0


# --------------------------------------------------- the binding on the device

def test_calls_go_to_the_current_stream():
    """The raw handle that the binding passes is the current stream's."""
    assert q._stream() == torch.cuda.current_stream().cuda_stream
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert q._stream() == side.cuda_stream
    assert q._stream(side) == side.cuda_stream
    assert q._stream() == torch.cuda.current_stream().cuda_stream != side.cuda_stream


def test_tensors_of_the_host_or_with_strides_are_refused():
    w, X = weight(1, 24, 32), tokens(2, 8, 32)
    off = offsets_of([4, 4])
    for call in (lambda: q.qlora_int8_linear_fwd(X.cpu(), w),
                 lambda: q.qlora_int8_linear_fwd(tokens(2, 32, 8).t(), w),
                 lambda: q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes.cpu(), w.scale, w.shape)),
                 lambda: q.qlora_int8_linear_fwd(X, w, Y=torch.zeros((8, 48), dtype=torch.bfloat16, device="cuda")[:, ::2]),
                 lambda: q.qlora_int8_expert_fwd(X, weight(3, 2, 24, 32), off.cpu()),
                 lambda: q.qlora_int8_expert_bwd(tokens(2, 8, 24).cpu(), weight(3, 2, 24, 32), off),
                 lambda: q.qlora_int8_quantize_rows(X.t())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.QloraError):
        q.qlora_int8_linear_fwd(tokens(2, 9, 8 * 32 + 1).flatten()[1:8 * 32 + 1].view(8, 32), w)  # not 16-byte aligned


@pytest.mark.parametrize("M", [2, 12, 300])
@pytest.mark.parametrize("K", [320, 8192])
def test_the_scales_are_taken_in_their_order(M, K):
    """Y = RN32(RN32(RN32(sum) x_scale) w_scale) to the bit, at either end of
    fp32: for tokens above FLT_MAX / (127 K) the first product may be infinite."""
    w = q.qlora_int8_quantize_rows(torch.randn((70, K), generator=gen(2), device="cuda") * 1e-3)
    for size in (1.0, 1e-37, 1e-34, 3e32, 1e35, 1e38):
        x = torch.rand((M, K), generator=gen(M), device="cuda") + 1
        x[1::2] *= -1
        X = (x * size).to(torch.bfloat16)
        xq = q.qlora_int8_quantize_rows(X)
        sums = (xq.codes.double() @ w.codes.double().T).float()  # below 2^53, rounded once
        want = (sums * xq.scale[:, None]) * w.scale
        Y = q.qlora_int8_linear_fwd(X, w, out_dtype=torch.float32)
        assert torch.equal(Y, want) and torch.equal(q.qlora_int8_linear_fwd(xq, w, out_dtype=torch.float32), want)
        assert torch.equal(q.qlora_int8_linear_fwd(X, w), want.to(torch.bfloat16))
        top = X.double().abs().max().item()
        assert want.isfinite().all() or top > ref.FLT_MAX / (127 * K)
