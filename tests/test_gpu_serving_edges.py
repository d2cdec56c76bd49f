"""GPU tests of the 8-bit serving path at the edges of what its documentation allows: alignments,
values that are not numbers, pages far apart in size, loose bounds, waits that run out, more than
one stream or thread. Oracles and derived tolerances as in test_gpu_kv.py and test_gpu_int8.py
unless a test derives its own.
"""

import time

import pytest
import torch

from test_gpu_kv import Setup
from rotation_bit_quantization_token_b200 import _lib, int8_matmul


pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (128, 64, True), (128, 128, False)])
def test_append_frequencies_at_any_element(D, rot, interleaved):
    """inv_freq may begin at any float of a larger array: the same bits as from an aligned copy."""
    s = Setup([3, 40], [5, 0], H=2, D=D, page=16, seed=70)
    batch = s.batch()
    k = torch.randn(43, 2, D, device="cuda").half()
    q = torch.randn(43, 6, D, device="cuda").half()
    table = torch.rand(rot // 2 + 3, device="cuda")
    for at in (1, 2, 3):
        part = table[at:at + rot // 2]
        assert part.data_ptr() % 16 == 4 * at % 16
        got, want = s.cache(), s.cache()
        a = got.append(k, k, *batch, q=q, inv_freq=part, interleaved=interleaved)
        b = want.append(k, k, *batch, q=q, inv_freq=part.clone(), interleaved=interleaved)
        assert torch.equal(a, b)
        assert torch.equal(got.k.view(torch.uint8), want.k.view(torch.uint8))
        assert torch.equal(got.k_scale, want.k_scale)


# ------------------------------------------------------------------------------------
# waits that run out
# ------------------------------------------------------------------------------------
def _product_gives_up(T, O, L):
    """A call whose loads are missing reports its waits within a few of their limits, and the same
    call afterwards is right."""
    lib = _lib.load()
    g = torch.Generator(device="cuda").manual_seed(T)
    a, w = (torch.randint(-128, 128, (n, L), generator=g, device="cuda", dtype=torch.int8) for n in (T, O))
    sa, sw = (torch.rand(n, generator=g, device="cuda") for n in (T, O))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = int8_matmul(a, sa, w, sw, status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert lib.fq_int8_debug_arm_stall(0.05) == _lib.FQ_OK
    t0 = time.monotonic()
    int8_matmul(a, sa, w, sw, status=st)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 2.0
    assert int(st) != 0
    st.zero_()
    for _ in range(3):
        assert torch.equal(int8_matmul(a, sa, w, sw, status=st), want)
    assert int(st) == 0


@pytest.mark.parametrize("T,O,L", [
    (3, 130, 144), (777, 513, 512),                                            # tiles of one CTA
    (5, 128, 8192), (20, 130, 8208), (64, 513, 6160), (100, 300, 8192), (333, 200, 9232)])  # K in 8, 8, 4, 8, 2 parts
def test_product_whose_waits_run_out(T, O, L):
    _product_gives_up(T, O, L)


@pytest.mark.parametrize("T,O,L", [(1990, 2100, 272), (300, 8200, 512), (2049, 2056, 4096)])
def test_pairs_whose_waits_run_out(T, O, L):
    """Pairs of CTAs: fewer stages than the ring holds, several tiles, long rows."""
    _product_gives_up(T, O, L)


def test_product_stall_hook_checks_its_limit():
    for bad in (0.0, -1.0, 11.0, float("nan")):
        assert _lib.load().fq_int8_debug_arm_stall(bad) == _lib.FQ_ERR_INVALID
