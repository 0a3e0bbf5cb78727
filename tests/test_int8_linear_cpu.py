"""The Int8 linear's refusals and marshalling on the CPU: argument errors of
the C entry points (nothing is launched on these paths), and the Python
binding's checks with a recorder in the library's place."""
import pytest
import torch

import bit_nf4_quantized_13_b200 as q
import int8_reference as ref
from test_binding_cpu import fake  # noqa: F401  (the recorder fixture)

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_13_b200 import build
    build.build()
    return q.lib


P = 1 << 20  # a 16-byte-aligned stand-in address; never dereferenced on these paths
BIG = 1 << 40


def test_quantize_rows_refusals(lib):
    f = lib.qlora_int8_quantize_rows
    assert f(P, 0, -1, 8, P, P, None, None) == INVALID
    assert f(P, 0, 4, 0, P, P, None, None) == INVALID
    assert f(P, 2, 4, 8, P, P, None, None) == INVALID            # unknown dtype
    assert f(P, 0, 4, 131073, P, P, None, None) == UNSUPPORTED
    assert f(P, 0, 1 << 31, 8, P, P, None, None) == UNSUPPORTED
    assert f(None, 1, 4, 8, P, P, None, None) == INVALID
    assert f(P + 2, 1, 4, 8, P, P, None, None) == INVALID
    assert f(P, 1, 4, 8, P + 8, P, None, None) == INVALID
    assert f(P, 1, 4, 8, P, None, None, None) == INVALID
    assert f(P, 1, 4, 8, P, P, P + 2, None) == INVALID           # misaligned status
    assert f(None, 1, 0, 8, None, None, None, None) == OK        # no rows: nothing enqueued


def test_linear_refusals(lib):
    for f, x, ws in ((lib.qlora_int8_linear_fwd, (P,), (P, BIG)), (lib.qlora_int8_matmul, (P, P), (P, BIG))):
        assert f(*x, -1, 8, 8, P, P, P, 1, *ws, None) == INVALID
        assert f(*x, 4, 0, 8, P, P, P, 1, *ws, None) == INVALID
        assert f(*x, 4, 8, 0, P, P, P, 1, *ws, None) == INVALID
        assert f(*x, 4, 8, 131073, P, P, P, 1, *ws, None) == UNSUPPORTED
        assert f(*x, 1 << 30, 8, 8, P, P, P, 1, *ws, None) == UNSUPPORTED
        assert f(*x, 4, 1 << 30, 8, P, P, P, 1, *ws, None) == UNSUPPORTED
        assert f(*x, 4, 8, 8, P, P, P, 2, *ws, None) == INVALID   # unknown output type
        assert f(*x, 4, 8, 8, P, P, P, -1, *ws, None) == INVALID
        assert f(*x, 4, 8, 8, None, P, P, 1, *ws, None) == INVALID
        assert f(*x, 4, 8, 8, P, P + 4, P, 1, *ws, None) == INVALID
        assert f(*x, 4, 8, 8, P, P, None, 1, *ws, None) == INVALID
        assert f(*(None,) * len(x), 4, 8, 8, P, P, P, 1, *ws, None) == INVALID
        assert f(*(None,) * len(x), 0, 8, 8, P, P, None, 1, None, 0, None) == OK  # no tokens
    assert lib.qlora_int8_matmul(P, P, 400, 64, 11008, P, P, P, 1, None, 0, None) == WORKSPACE  # a split contraction
    f = lib.qlora_int8_linear_fwd
    assert f(P, 400, 8, 8, P, P, P, 1, None, BIG, None) == WORKSPACE
    assert f(P, 400, 8, 8, P, P, P, 1, P + 8, BIG, None) == WORKSPACE
    assert f(P, 400, 8, 8, P, P, P, 1, P, 100, None) == WORKSPACE
    f = lib.qlora_int8_linear_bwd
    assert f(P, -1, 8, 8, P, P, P, P, BIG, None) == INVALID
    assert f(P, 4, 8, 131073, P, P, P, P, BIG, None) == UNSUPPORTED
    assert f(None, 4, 8, 8, P, P, P, P, BIG, None) == INVALID
    assert f(P, 4, 8, 8, P, P, P + 2, P, BIG, None) == INVALID
    assert f(P, 4, 8, 8, None, P, P, P, BIG, None) == INVALID
    assert f(P, 400, 9, 8, P, P, P, None, 0, None) == WORKSPACE  # rows of dY to be padded
    assert f(None, 0, 8, 8, P, P, None, None, 0, None) == OK


def test_expert_refusals(lib):
    for f, x, ws in ((lib.qlora_int8_expert_fwd, (P,), (P, BIG)), (lib.qlora_int8_expert_matmul, (P, P), (P, BIG))):
        assert f(*x, P, 4, 0, 8, 8, P, P, P, 1, *ws, None) == INVALID
        assert f(*x, P, 4, 1025, 8, 8, P, P, P, 1, *ws, None) == UNSUPPORTED
        assert f(*x, P, 4, 1024, 1 << 22, 8, P, P, P, 1, *ws, None) == UNSUPPORTED  # E N >= 2^31
        assert f(*x, None, 4, 2, 8, 8, P, P, P, 1, *ws, None) == INVALID            # no offsets
        assert f(*x, P + 4, 4, 2, 8, 8, P, P, P, 1, *ws, None) == INVALID
        assert f(*x, None, 0, 2, 8, 8, P, P, None, 1, None, 0, None) == OK
    assert lib.qlora_int8_expert_fwd(P, P, 400, 2, 8, 8, P, P, P, 1, P, 0, None) == WORKSPACE
    f = lib.qlora_int8_expert_bwd
    assert f(P, None, 4, 2, 8, 8, P, P, P, P, BIG, None) == INVALID
    assert f(P, P, 4, 1025, 8, 8, P, P, P, P, BIG, None) == UNSUPPORTED
    assert f(P, P, 4, 2, 8, 8, P, P, None, P, BIG, None) == INVALID
    assert f(P, P, 0, 2, 8, 8, P, P, None, None, 0, None) == OK


def test_overlapping_arrays_are_refused(lib):
    A = [(i + 1) << 40 for i in range(7)]  # far apart; every call below has one overlap and is refused for it
    X, W, S, Y, WS, O, XS = A
    T, N, K = 40, 64, 96
    f = lib.qlora_int8_linear_fwd
    for y, ws in ((X, WS), (X + T * K * 2 - 16, WS), (W + 16, WS), (S, WS), (WS, WS), (Y, Y), (Y, X), (Y, W), (Y, S),
                  (X - T * N * 2 + 16, WS)):
        assert f(X, T, N, K, W, S, y, 1, ws, 1 << 30, None) == INVALID
    assert f(X, 2, N, K, W, S, X, 1, None, 0, None) == INVALID  # one kernel, no workspace
    assert lib.qlora_int8_matmul(X, XS, T, N, K, W, S, XS, 1, WS, 1 << 30, None) == INVALID
    assert lib.qlora_int8_expert_fwd(X, O, T, 2, N, K, W, S, O, 1, WS, 1 << 30, None) == INVALID
    f = lib.qlora_int8_linear_bwd
    for n, dx, ws in ((N, X, WS), (N, W, WS), (N, S, WS), (63, Y, X), (63, Y, Y), (63, Y, W)):
        assert f(X, T, n, K, W, S, dx, ws, 1 << 30, None) == INVALID
    f = lib.qlora_int8_quantize_rows
    for codes, scale, status in ((X, S, None), (X + T * K * 2 - 16, S, None), (W, W, None), (W, X, None), (W, S, W),
                                 (W, S, S), (W, S, X)):
        assert f(X, 1, T, K, codes, scale, status, None) == INVALID


def test_workspace_sizes(lib):
    # the tokens' codes (rows of 16-byte multiples) and scales at least
    assert q.qlora_int8_linear_fwd_workspace_size(100, 8, 33) >= 100 * 48 + 400
    assert q.qlora_int8_expert_fwd_workspace_size(100, 4, 8, 33) >= 100 * 48 + 400
    assert q.qlora_int8_linear_fwd_workspace_size(4, 8, 131073) == 0
    assert q.qlora_int8_expert_bwd_workspace_size(4, 1025, 8, 8) == 0
    assert q.qlora_int8_matmul_workspace_size(1, 64, 4096) == 0
    assert q.qlora_int8_expert_matmul_workspace_size(400, 4, 8, 33) < q.qlora_int8_expert_fwd_workspace_size(400, 4, 8, 33)
    assert q.qlora_int8_linear_bwd_workspace_size(100, 40, 64) == 0
    assert q.qlora_int8_linear_bwd_workspace_size(100, 33, 64) >= 100 * 40 * 2  # padded rows of dY
    # few tiles with a long contraction: the parts' sums
    assert q.qlora_int8_linear_bwd_workspace_size(100, 8192, 64) >= 2 * 128 * 256 * 4
    assert q.qlora_int8_matmul_workspace_size(100, 64, 11008) >= 2 * 128 * 256 * 4
    assert q.qlora_int8_linear_bwd_workspace_size(0, 64, 64) == 0
    assert q.qlora_int8_linear_fwd_workspace_size(1, 64, 4096) == 0  # one kernel that quantizes its own token


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_operands_reach_the_library(fake):  # noqa: F811
    w, we = q.alloc_int8_rows((24, 33), "cpu"), q.alloc_int8_rows((3, 24, 33), "cpu")
    assert w.codes.shape == (24, 48) and we.codes.shape == (3, 24, 48) and we.scale.shape == (3, 24)
    assert w.nbytes() == 24 * 48 + 24 * 4
    off = torch.zeros(4, dtype=torch.int32)
    Y = q.qlora_int8_linear_fwd(bf16(5, 33), w)
    name, args = fake.calls[-1]
    assert name == "qlora_int8_linear_fwd" and args[1:4] == (5, 24, 33) and args[7] == 1
    assert Y.shape == (5, 24) and Y.dtype == torch.bfloat16
    Y = q.qlora_int8_linear_fwd(q.alloc_int8_rows((5, 33), "cpu"), w, out_dtype=torch.float32)
    name, args = fake.calls[-1]
    assert name == "qlora_int8_matmul" and args[2:5] == (5, 24, 33) and args[8] == 0 and Y.dtype == torch.float32
    q.qlora_int8_linear_fwd(bf16(5, 33), w, Y=torch.zeros(5, 24))  # the output's own type is taken
    assert fake.calls[-1][1][7] == 0
    assert q.qlora_int8_linear_bwd(bf16(5, 24), w).shape == (5, 33)
    assert fake.calls[-1][0] == "qlora_int8_linear_bwd" and fake.calls[-1][1][1:4] == (5, 24, 33)
    assert q.qlora_int8_expert_fwd(bf16(5, 33), we, off).shape == (5, 24)
    assert fake.calls[-1][0] == "qlora_int8_expert_fwd" and fake.calls[-1][1][2:6] == (5, 3, 24, 33)
    q.qlora_int8_expert_fwd(q.alloc_int8_rows((5, 33), "cpu"), we, off)
    assert fake.calls[-1][0] == "qlora_int8_expert_matmul" and fake.calls[-1][1][3:7] == (5, 3, 24, 33)
    assert q.qlora_int8_expert_bwd(bf16(5, 24), we, off).shape == (5, 33)
    assert fake.calls[-1][0] == "qlora_int8_expert_bwd" and fake.calls[-1][1][2:6] == (5, 3, 24, 33)
    r = q.qlora_int8_quantize_rows(torch.zeros(2, 3, 33))
    assert r.shape == (2, 3, 33) and r.codes.shape == (2, 3, 48)
    assert fake.calls[-1][0] == "qlora_int8_quantize_rows" and fake.calls[-1][1][1:4] == (0, 6, 33)


def test_disagreeing_operands_are_refused(fake):  # noqa: F811
    w, we = q.alloc_int8_rows((24, 33), "cpu"), q.alloc_int8_rows((3, 24, 33), "cpu")
    off = torch.zeros(4, dtype=torch.int32)
    X, dY = bf16(5, 33), bf16(5, 24)
    bad = [
        lambda: q.qlora_int8_linear_fwd(bf16(5, 48), w),                            # K
        lambda: q.qlora_int8_linear_fwd(X.float(), w),                              # dtype
        lambda: q.qlora_int8_linear_fwd(X, we),                                     # a weight of experts
        lambda: q.qlora_int8_linear_fwd(X[0], w),                                   # not 2-D
        lambda: q.qlora_int8_linear_fwd(X, w, out_dtype=torch.float16),
        lambda: q.qlora_int8_linear_fwd(X, w, Y=bf16(5, 25)),
        lambda: q.qlora_int8_linear_fwd(X, w, out_dtype=torch.float32, Y=bf16(5, 24)),
        lambda: q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes[:, :33], w.scale, (24, 33))),   # rows not padded
        lambda: q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes, w.scale[:5], (24, 33))),
        lambda: q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes.to(torch.uint8), w.scale, (24, 33))),
        lambda: q.qlora_int8_linear_fwd(X, q.Int8Rows(w.codes, w.scale.double(), (24, 33))),
        lambda: q.qlora_int8_linear_fwd(q.alloc_int8_rows((5, 34), "cpu"), w),
        lambda: q.qlora_int8_linear_bwd(X, w),                                      # N
        lambda: q.qlora_int8_linear_bwd(q.alloc_int8_rows((5, 24), "cpu"), w),      # quantized gradients
        lambda: q.qlora_int8_linear_bwd(dY, w, dX=bf16(5, 48)),
        lambda: q.qlora_int8_linear_bwd(dY, w, dX=torch.zeros(5, 33)),
        lambda: q.qlora_int8_expert_fwd(X, w, off),                                 # a dense weight
        lambda: q.qlora_int8_expert_fwd(X, we, off[:3]),
        lambda: q.qlora_int8_expert_fwd(X, we, off.long()),
        lambda: q.qlora_int8_expert_fwd(X, we, None),
        lambda: q.qlora_int8_expert_bwd(dY, we, None),
        lambda: q.qlora_int8_expert_bwd(dY, we, off.float()),
        lambda: q.qlora_int8_quantize_rows(X.half()),
        lambda: q.qlora_int8_quantize_rows(X[0]),
        lambda: q.qlora_int8_quantize_rows(bf16(5, 0)),
        lambda: q.qlora_int8_quantize_rows(X, out=q.alloc_int8_rows((5, 34), "cpu")),
        lambda: q.qlora_int8_quantize_rows(X, status=torch.zeros(1, dtype=torch.int64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert fake.calls == [], "nothing may reach the library"


def test_library_status_becomes_an_exception(fake):  # noqa: F811
    fake.status = 2
    with pytest.raises(q.QloraError) as e:
        q.qlora_int8_linear_fwd(bf16(5, 33), q.alloc_int8_rows((24, 33), "cpu"))
    assert e.value.status == 2


def test_zero_rows_refusals(lib):
    f = lib.qlora_int8_expert_zero_rows
    assert f(P, -1, 2, 8, 1, P, None) == INVALID
    assert f(P, 4, 0, 8, 1, P, None) == INVALID
    assert f(P, 4, 2, 0, 1, P, None) == INVALID
    assert f(P, 4, 2, 8, 2, P, None) == INVALID                 # unknown type
    assert f(P, 4, 1025, 8, 1, P, None) == UNSUPPORTED
    assert f(P, 1 << 30, 2, 8, 1, P, None) == UNSUPPORTED
    assert f(None, 4, 2, 8, 1, P, None) == INVALID
    assert f(P + 4, 4, 2, 8, 1, BIG, None) == INVALID
    assert f(P, 4, 2, 8, 1, None, None) == INVALID
    assert f(P, 4, 2, 8, 1, BIG + 2, None) == INVALID
    assert f(P, 4, 2, 8, 1, P, None) == INVALID                 # the offsets lie in the output
    assert f(P + 48, 4, 2, 8, 1, P, None) == INVALID
    assert f(None, 0, 2, 8, 1, None, None) == OK


def test_only_outputs_made_by_an_expert_call_are_cleared(fake):  # noqa: F811
    w, we, off = q.alloc_int8_rows((24, 33), "cpu"), q.alloc_int8_rows((3, 24, 33), "cpu"), torch.zeros(4, dtype=torch.int32)
    names = lambda: [c[0] for c in fake.calls if not c[0].endswith("_workspace_size")]  # noqa: E731
    q.qlora_int8_expert_fwd(bf16(5, 33), we, off, out_dtype=torch.float32)
    assert names() == ["qlora_int8_expert_zero_rows", "qlora_int8_expert_fwd"]
    assert fake.calls[-2][1][1:5] == (5, 3, 24, 0) and fake.calls[-2][1][5] == fake.calls[-1][1][8]
    fake.calls.clear()
    q.qlora_int8_expert_fwd(q.alloc_int8_rows((5, 33), "cpu"), we, off)
    assert names() == ["qlora_int8_expert_zero_rows", "qlora_int8_expert_matmul"]
    fake.calls.clear()
    q.qlora_int8_expert_bwd(bf16(5, 24), we, off)
    assert names() == ["qlora_int8_expert_zero_rows", "qlora_int8_expert_bwd"]
    assert fake.calls[-2][1][1:5] == (5, 3, 33, 1) and fake.calls[-2][1][5] == fake.calls[-1][1][8]
    fake.calls.clear()
    q.qlora_int8_expert_fwd(bf16(5, 33), we, off, Y=bf16(5, 24))
    q.qlora_int8_expert_bwd(bf16(5, 24), we, off, dX=bf16(5, 33))
    q.qlora_int8_linear_fwd(bf16(5, 33), w)
    q.qlora_int8_linear_bwd(bf16(5, 24), w)
    assert "qlora_int8_expert_zero_rows" not in names()


# The gradient tests' own checks, fed with right and with wrong gradients.

def small_gradient():
    g = torch.Generator()
    g.manual_seed(5)
    M, N, K = 40, 264, 320
    codes, scale, _ = ref.quantize_rows(torch.randn((N, K), generator=g) * 0.02)
    W = ref.compute_weight(codes, scale)
    dY = (torch.randn((M, N), generator=g) * 0.1).to(torch.bfloat16)
    X = torch.randn((M, K), generator=g, dtype=torch.float64)
    picks = torch.stack([torch.randint(0, n, (120,), generator=g) for n in (M, K)], 1).tolist()
    return dY, codes, scale, W, X, picks + [[m, k] for m in (0, M - 1) for k in (0, K - 1)]


def bf16_product(dY, W):
    return (dY.float() @ W.float()).to(torch.bfloat16)


def test_the_difference_check_rejects_wrong_gradients():
    dY, codes, scale, W, X, picks = small_gradient()
    good = bf16_product(dY, W)
    ref.check_differences(good, dY, W, X, picks)
    zero_row, zero_column = good.clone(), good.clone()
    zero_row[picks[0][0]], zero_column[:, picks[1][1]] = 0, 0
    wrong = {"scaled by 0.99": (bf16_product(dY, W).float() * 0.99).to(torch.bfloat16), "a row of zeros": zero_row,
             "a column of zeros": zero_column, "the last term dropped": bf16_product(dY[:, :-1], W[:-1]),
             "a token's neighbour": good.roll(1, 0), "a column's neighbour": good.roll(1, 1),
             "the scales dropped": bf16_product(dY, codes)}
    for name, dX in wrong.items():
        with pytest.raises(AssertionError):
            ref.check_differences(dX, dY, W, X, picks)
            pytest.fail(f"accepted: {name}")


@pytest.mark.parametrize("M,N,K", [(16, 11008, 48), (5, 4097, 70), (3, 16500, 20)])
def test_the_exact_checks_reject_wrong_gradients(M, N, K):
    g = torch.Generator()
    g.manual_seed(N)
    dY, codes, scale = ref.integer_gradient(g, M, N, K)
    W = codes.double() * scale.double()[:, None]
    want = ref.exact_gradient(dY, codes, scale)
    assert torch.equal(bf16_product(dY, W), want)  # fp32 sums in torch's order: exact too
    assert (dY.double().abs() @ W.abs()).max() < 2 ** 24
    for lost in (0, 63, 64, N // 2, N - 1):
        part = dY.clone()
        part[:, lost] = 0
        assert dY[:, lost].any() and not torch.equal(bf16_product(part, W), want), lost
    codes, scale, _ = ref.quantize_rows(torch.randn((300, K), generator=g) * 0.02)
    held = ref.round32(codes * scale[:, None]).float()
    cut = (held.view(torch.int32) & -65536).view(torch.float32)  # W' truncated to bf16
    assert not torch.equal(cut.to(torch.bfloat16), ref.compute_weight(codes, scale).to(torch.bfloat16))
