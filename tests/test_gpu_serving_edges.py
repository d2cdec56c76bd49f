"""GPU tests of the 8-bit serving path at the edges of what its documentation allows: alignments,
values that are not numbers, pages far apart in size, loose bounds, waits that run out, more than
one stream or thread. Oracles and derived tolerances as in test_gpu_kv.py and test_gpu_int8.py
unless a test derives its own.
"""

import pytest
import torch

from test_gpu_kv import Setup


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
