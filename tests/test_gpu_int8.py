"""GPU tests of the INT8 path: the per-token quantizer's INT8 codes and fq_int8_matmul, against
float64.

Tolerances, derived from the arithmetic:
* product: the integer sum is exact; float32(sum), the two multiplications by scales and the
  final rounding are off by at most half a step each, so |C - ref| <= (3 * 2^-24 + h)(1 + 2^-7)
  |ref| with h = 0 (fp32), 2^-8 (bf16) or 2^-11 (fp16, normal range; 2^-25 absolute below it).
* codes: x'' is a float32 sum of M + N exact products with its intermediate held to 22 bits:
  |dx''| <= E = ((M + N) 2^-23 + 2^-21) (|P1| |x| |P2|). A code is x'' / s rounded to an integer
  (half a unit), s and its reciprocal good to E_max / amax + 2^-22 relative.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from rotation_bit_quantization_token_b200 import FQError, FlatQuant, int8_matmul
from rotation_bit_quantization_token_b200.workloads import random_orthogonal

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _close(C, ref, dt):
    tol = (3 * 2.0 ** -24 + HALF[dt]) * (1 + 2.0 ** -7) * np.abs(ref) + (2.0 ** -25 if dt is torch.float16 else 0)
    err = np.abs(C.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


def _operands(T, O, L, seed, lo=-128, hi=127):
    g = np.random.default_rng([seed, T, O, L])
    a = g.integers(lo, hi + 1, (T, L), dtype=np.int8)
    w = g.integers(lo, hi + 1, (O, L), dtype=np.int8)
    return a, (0.5 + g.random(T)).astype(np.float32) * 2.0 ** -6, w, (0.5 + g.random(O)).astype(np.float32) * 2.0 ** -8


def _dev(*arrays):
    return [torch.from_numpy(x).cuda() for x in arrays]


# every token-tile width and its neighbours, ragged channels, K down to 16 codes, K tails of 16
SHAPES = [(1, 1, 16), (1, 128, 4096), (3, 130, 144), (16, 300, 2048), (17, 64, 4112), (32, 1000, 1024),
          (33, 257, 2064), (64, 129, 8192), (65, 384, 512), (128, 255, 1040), (129, 640, 4096), (300, 1030, 1552),
          (777, 513, 2048), (2, 5000, 16384), (1000, 3, 96),
          # pairs of CTAs: one tile each, several each (aligned and unaligned rows of C), long K
          (1990, 2100, 272), (300, 8200, 512), (2600, 3001, 144), (2600, 3008, 400), (2049, 2056, 4096)]


@pytest.mark.parametrize("T,O,L", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_product_matches_exact_sums(T, O, L, dt):
    a, sa, w, sw = _operands(T, O, L, 1)
    A, SA, W, SW = _dev(a, sa, w, sw)
    out = torch.full((T + 2, O), float("nan"), dtype=dt, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = int8_matmul(A, SA, W, SW, out_dtype=dt, out=out[1:T + 1], status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    _close(got, osv.int8_matmul(a, sa, w, sw), dt)
    assert torch.isnan(out[0]).all() and torch.isnan(out[T + 1]).all()  # nothing beside C is written


def test_extreme_sums_are_exact():
    """All codes -128 over the longest row: the sum is 65536 * 2^14 = 2^30, exact in int32."""
    L = 65536
    A = torch.full((20, L), -128, dtype=torch.int8, device="cuda")
    W = torch.full((140, L), -128, dtype=torch.int8, device="cuda")
    W[1] = 127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    C = int8_matmul(A, one(20), W, one(140), out_dtype=torch.float32).cpu()
    assert torch.all(C[:, 0] == 2.0 ** 30) and torch.all(C[:, 1] == -128.0 * 127 * 65536) and torch.all(C[:, 139] == 2.0 ** 30)


def test_scales_zero_negative_and_special():
    a, sa, w, sw = _operands(5, 130, 256, 2)
    sa[0], sa[1], sw[3] = 0.0, -1.5, np.inf
    A, SA, W, SW = _dev(a, sa, w, sw)
    C = int8_matmul(A, SA, W, SW, out_dtype=torch.float32).cpu().numpy()
    acc = a.astype(np.int64) @ w.astype(np.int64).T
    keep = np.arange(130) != 3
    assert np.all(C[0][keep] == 0) and np.isnan(C[0, 3])
    ref = osv.int8_matmul(a, sa, w, np.where(keep, sw, 1))[1:][:, keep]
    assert np.all(np.abs(C[1:][:, keep] - ref) <= 3.1 * 2.0 ** -24 * np.abs(ref))
    want = np.sign(acc[1:, 3]) * np.sign(sa[1:]) * np.inf
    assert np.array_equal(C[1:, 3][acc[1:, 3] != 0], want[acc[1:, 3] != 0])


def test_split_sums_do_not_depend_on_the_run():
    a, sa, w, sw = _operands(7, 400, 8192, 3)
    A, SA, W, SW = _dev(a, sa, w, sw)
    first = int8_matmul(A, SA, W, SW)
    for _ in range(5):
        assert torch.equal(int8_matmul(A, SA, W, SW), first)


def test_large_output_offsets():
    """T * O past 2^31 elements: the last rows against exact sums."""
    T, O, L = 262144, 8200, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    A = torch.randint(-128, 128, (T, L), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (O, L), generator=g, device="cuda", dtype=torch.int8)
    C = int8_matmul(A, torch.ones(T, device="cuda"), W, torch.ones(O, device="cuda"), out_dtype=torch.float16)
    rows = [0, 1, 131071, 262000, T - 2, T - 1]
    ref = A[rows].double().cpu().numpy() @ W.double().cpu().numpy().T
    got = C[rows].double().cpu().numpy()
    fits = np.abs(ref) < 65000
    assert np.all(np.abs(got - ref)[fits] <= 2.0 ** -11 * np.abs(ref)[fits])


def test_other_stream_and_graph():
    a, sa, w, sw = _operands(40, 600, 2048, 4)
    A, SA, W, SW = _dev(a, sa, w, sw)
    want = int8_matmul(A, SA, W, SW)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    int8_matmul(A, SA, W, SW, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = int8_matmul(A, SA, W, SW)
    A.copy_(A.flip(0))
    SA.copy_(SA.flip(0))
    graph.replay()
    assert torch.equal(captured, want.flip(0))


def test_refusals():
    a, sa, w, sw = _operands(4, 6, 64, 6)
    A, SA, W, SW = _dev(a, sa, w, sw)
    for bad in [lambda: int8_matmul(A.to(torch.uint8), SA, W, SW), lambda: int8_matmul(A, SA.double(), W, SW),
                lambda: int8_matmul(A, SA[:3], W, SW), lambda: int8_matmul(A[:, :32].contiguous(), SA, W, SW),
                lambda: int8_matmul(A.t(), SA, W, SW), lambda: int8_matmul(A, SA, W, SW, out_dtype=torch.int32),
                lambda: int8_matmul(A, SA, W, SW, out=torch.empty(4, 5, dtype=torch.bfloat16, device="cuda")),
                lambda: int8_matmul(A[0], SA, W, SW)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(FQError):
        int8_matmul(A[:, :8].contiguous(), SA, W[:, :8].contiguous(), SW)  # L % 16
    with pytest.raises(FQError):
        int8_matmul(A[:0], SA[:0], W, SW)


# ---- INT8 codes of the per-token quantizer ----

def _check_codes(K, M, N, clip, dtype, kernel, seed=0):
    g = np.random.default_rng([seed, K, M, N])
    x = torch.from_numpy(g.standard_normal((K, M, N), dtype=np.float32))
    x.view(K, -1)[:, g.integers(0, M * N, 3)] *= 20
    x[K // 2] = 0.0
    x = x.to(dtype)
    P1 = torch.from_numpy(random_orthogonal(M, seed, 2)).to(dtype)
    P2 = torch.from_numpy(random_orthogonal(N, seed, 3)).to(dtype)
    h = FlatQuant(K, M, N, dtype, kernel=kernel)
    codes, qs = h.quantize_per_token(x.cuda(), P1.cuda(), P2.cuda(), clip_ratio=clip, out_dtype="int8")
    torch.cuda.synchronize()
    assert h.device_status() == 0 and (kernel == "auto" or h.last_kernel == kernel)
    f = lambda t: t.double().numpy()  # noqa: E731
    ref, rqs, v = osv.per_token_quantize8(oracle.rotate(f(x), f(P1), f(P2)), clip)
    mag = np.matmul(np.abs(f(P1)), np.matmul(np.abs(f(x)), np.abs(f(P2)))).reshape(K, -1)
    E = ((M + N) * 2.0 ** -23 + 2.0 ** -21) * mag
    amax = np.maximum(rqs * 127 / clip, 1e-30)
    rel = E.max(axis=1) / amax + 2.0 ** -22
    got, gqs = codes.cpu().numpy().astype(np.int64), qs.double().cpu().numpy()
    assert np.all(np.abs(gqs - rqs) <= rel * rqs)
    s = np.where(rqs > 0, rqs, 1.0)[:, None]
    off = np.abs(got - np.clip(v, -128, 127)) - 0.5
    assert np.all(off <= E / s + np.abs(v) * rel[:, None]), float(off.max())
    assert np.all(got[K // 2] == 0) and gqs[K // 2] == 0
    assert np.mean(got != ref) < 1e-3


@pytest.mark.parametrize("K,M,N", [(3, 16, 16), (5, 7, 11), (37, 3, 33), (9, 40, 72), (4, 256, 250)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_int8_codes_general(K, M, N, dtype):
    _check_codes(K, M, N, 0.95, dtype, "general")


@pytest.mark.parametrize("K,M,N", [(2, 64, 64), (301, 64, 128), (333, 128, 112), (150, 128, 128), (613, 32, 80),
                                   (450, 64, 96), (305, 128, 80), (700, 64, 64), (400, 128, 96)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_int8_codes_tensor_core(K, M, N, dtype):
    _check_codes(K, M, N, 1.0, dtype, "tcgen05")


@pytest.mark.parametrize("kernel,M,N", [("general", 16, 16), ("tcgen05", 64, 64), ("tcgen05", 128, 112), ("tcgen05", 128, 128)])
def test_int8_ties_and_clamp_are_exact(kernel, M, N):
    """With identity rotations x'' = x; a token whose maximum is 127 * 2^-3 has quantScale 2^-3
    exactly, and every half-integer multiple of it rounds to even; with clipRatio 127 / 200 (as a
    float64 quotient) large values clamp to 127 and -128."""
    K = 5
    g = np.random.default_rng(7)
    half = g.integers(-253, 254, (K, M * N)) / 2.0
    half[:, 0], half[:, 1] = 127.0, -127.0
    x = torch.from_numpy(half / 8).to(torch.bfloat16).reshape(K, M, N)
    assert np.array_equal(x.double().numpy().reshape(K, -1) * 8, half)
    I1, I2 = torch.eye(M, dtype=torch.bfloat16).cuda(), torch.eye(N, dtype=torch.bfloat16).cuda()
    h = FlatQuant(K, M, N, torch.bfloat16, kernel=kernel)
    codes, qs = h.quantize_per_token(x.cuda(), I1, I2, out_dtype="int8")
    assert np.array_equal(qs.cpu().numpy(), np.full(K, 0.125, dtype=np.float32))
    assert np.array_equal(codes.cpu().numpy(), np.rint(half).astype(np.int8))
    codes, qs = h.quantize_per_token(x.cuda(), I1, I2, clip_ratio=0.5, out_dtype="int8")  # scale 2^-4
    assert np.array_equal(qs.cpu().numpy(), np.full(K, 0.0625, dtype=np.float32))
    assert np.array_equal(codes.cpu().numpy(), np.clip(2 * half, -128, 127).astype(np.int8))


def test_int8_output_checks():
    h = FlatQuant(4, 16, 16)
    x = torch.zeros(4, 16, 16, dtype=torch.bfloat16, device="cuda")
    P = torch.eye(16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="bytes"):
        h.quantize_per_token(x, P, P, out_dtype="int8", out=torch.empty(4, 128, dtype=torch.int8, device="cuda"))
    out = torch.empty(4, 256, dtype=torch.int8, device="cuda")
    assert h.quantize_per_token(x, P, P, out_dtype="int8", out=out)[0] is out


@pytest.mark.parametrize("K,M,N,O", [(16, 64, 64, 384), (200, 128, 112, 257)])
def test_rotated_linear_layer(K, M, N, O):
    """Quantizer and product together: the product of the codes and scales that the quantizer
    gave, exactly; and near the unquantized product, by the codes' half step."""
    g = np.random.default_rng([K, M, N, O])
    x = torch.from_numpy(g.standard_normal((K, M, N), dtype=np.float32)).to(torch.bfloat16)
    P1 = torch.from_numpy(random_orthogonal(M, 1, 2)).to(torch.bfloat16)
    P2 = torch.from_numpy(random_orthogonal(N, 1, 3)).to(torch.bfloat16)
    w = g.integers(-127, 128, (O, M * N), dtype=np.int8)
    sw = (g.random(O) + 0.5).astype(np.float32) * 1e-3
    codes, qs = FlatQuant(K, M, N).quantize_per_token(x.cuda(), P1.cuda(), P2.cuda(), out_dtype="int8")
    C = int8_matmul(codes, qs, *_dev(w, sw), out_dtype=torch.float32)
    a, s = codes.cpu().numpy(), qs.cpu().numpy()
    _close(C, osv.int8_matmul(a, s, w, sw), torch.float32)
    f = lambda t: t.double().numpy()  # noqa: E731
    full = oracle.rotate(f(x), f(P1), f(P2)).reshape(K, -1) @ (w.astype(np.float64) * sw[:, None].astype(np.float64)).T
    bound = 0.51 * s[:, None] * np.abs(w.astype(np.float64)).sum(1)[None, :] * sw[None, :]
    assert np.all(np.abs(C.double().cpu().numpy() - full) <= bound)


@pytest.mark.parametrize("T,O,L", [(5, 128, 8192), (20, 130, 8208), (40, 100, 4096), (64, 513, 6160), (100, 300, 8192),
                                   (200, 128, 4112), (333, 200, 9232)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_product_of_split_tiles(T, O, L, dt):
    """Few tiles of long rows: K is divided among the CTAs of a cluster, up to eight."""
    test_product_matches_exact_sums(T, O, L, dt)


@pytest.mark.parametrize("T,O,L", [(130, 100, 1040), (192, 257, 4112), (333, 300, 8192), (384, 6200, 528), (570, 129, 2064)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_product_of_middle_tiles(T, O, L, dt):
    """Token counts that pad less in tiles of 192, whole and split."""
    test_product_matches_exact_sums(T, O, L, dt)
