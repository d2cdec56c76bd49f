"""GPU tests of the 8-bit serving path at the edges of what its documentation allows: alignments,
values that are not numbers, pages far apart in size, loose bounds, waits that run out, more than
one stream or thread. Oracles and derived tolerances as in test_gpu_kv.py and test_gpu_int8.py
unless a test derives its own.
"""

import threading
import time

import numpy as np
import pytest
import torch

from oracle import serving as osv
from test_gpu_kv import HALF, Setup, _check_append, _check_attention, f64
from rotation_bit_quantization_token_b200 import (FlatQuant, HostPipeline, KVCache, _lib, int8_device_status,
                                                  int8_matmul, quantize_mx_static)

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


@pytest.mark.parametrize("T,O,L", [(3, 130, 144), (5, 128, 8192), (2049, 2056, 4096)])
def test_waits_that_run_out_are_kept_without_a_status_tensor(T, O, L):
    a, w = (torch.ones(n, L, dtype=torch.int8, device="cuda") for n in (T, O))
    sa, sw = (torch.ones(n, device="cuda") for n in (T, O))
    int8_matmul(a, sa, w, sw)
    assert int8_device_status() == 0
    assert _lib.load().fq_int8_debug_arm_stall(0.05) == _lib.FQ_OK
    int8_matmul(a, sa, w, sw)
    assert int8_device_status() != 0 and int8_device_status() == 0
    assert torch.all(int8_matmul(a, sa, w, sw, out_dtype=torch.float32) == L) and int8_device_status() == 0
    assert _lib.load().fq_int8_device_status(None) == _lib.FQ_ERR_NULLPTR


def test_product_stall_hook_checks_its_limit():
    for bad in (0.0, -1.0, 11.0, float("nan")):
        assert _lib.load().fq_int8_debug_arm_stall(bad) == _lib.FQ_ERR_INVALID


# ------------------------------------------------------------------------------------
# attention over codes that are not numbers
# ------------------------------------------------------------------------------------
def _with_nans(s, at):
    """NaN codes in live tokens: (sequence, position, "k" or "v", head, element)."""
    for b, pos, which, h, d in at:
        (s.k if which == "k" else s.v)[s.table[b, pos // s.page], h, pos % s.page, d] = 0x7F + 0x80 * (d % 2)
    return s


def _check_nan_attention(s, dtype, G, causal=True, max_seq_len=None):
    """Outputs and lse are NaN exactly where the formula's are (a row sees a NaN key; an element sees
    a NaN value), and elsewhere within the tolerance of test_gpu_kv.py."""
    Hq, D, n = s.H * G, s.D, s.cu[-1]
    q = torch.randn(n, Hq, D, generator=torch.Generator().manual_seed(9)).to(dtype).cuda()
    cache, scale, keys = s.cache(), D ** -0.5, max(s.lens)
    out, lse = cache.attention(q, *s.batch(), max_q_len=max(s.new), max_seq_len=max_seq_len or keys, scale=scale,
                               causal=causal, return_lse=True)
    assert cache.device_status() == 0
    ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, scale, causal)
    assert np.isnan(ro).any() and not np.isnan(ro).all()
    assert np.array_equal(np.isnan(f64(lse)), np.isnan(rl))
    assert np.array_equal(np.isnan(f64(out)), np.isnan(ro))
    vmax = np.nanmax(np.abs(osv.E4M3)) * np.exp2(s.vs.max() - 127.0)
    e = (D * 2.0 ** -23 + 2.0 ** -21) * np.nan_to_num(info["a"])
    tol = ((2 * e + 2.0 ** -11 + (keys + 66) * 2.0 ** -23)[..., None] * info["pv"] + keys * 2.0 ** -25 * vmax
           + HALF[dtype] * np.abs(ro) + 2.0 ** -25)
    fine = ~np.isnan(ro)
    assert np.all(np.abs(f64(out) - ro)[fine] <= tol[fine])
    ltol = e + (keys + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(np.nan_to_num(rl)))
    fine = ~np.isnan(rl)
    assert np.all(np.abs(f64(lse) - rl)[fine] <= ltol[fine])


@pytest.mark.parametrize("new,ctx,G,longest", [
    ([1, 1, 1], [300, 40, 700], 4, None),        # decode steps: one CTA or a cluster a sequence
    ([1, 1, 1], [300, 40, 700], 4, 200000),      # chunks through the workspace
    ([90, 100], [300, 256], 1, None)])           # prompts
def test_nan_key_that_every_row_sees(new, ctx, G, longest):
    """A NaN key among the first: the outputs of the rows that see it and their lse are NaN, not an
    lse of a row that sees nothing."""
    width = -(-(longest or 1) // 64)
    s = Setup(new, ctx, H=2, D=128, page=64, seed=71, width=max(width, 16)).fill()
    _check_nan_attention(_with_nans(s, [(0, 5, "k", 1, 3), (1, 0, "k", 0, 127)]), torch.bfloat16, G, max_seq_len=longest)


@pytest.mark.parametrize("D,page,G", [(128, 64, 1), (64, 16, 4), (128, 32, 2)])
def test_nan_keys_wherever_they_lie(D, page, G):
    """NaN keys of cached and of new tokens, in whole steps and in the last, incomplete one of a prompt:
    rows before them stay numbers, rows from them on are NaN."""
    s = Setup([90, 70, 3], [300, 5, 200], H=2, D=D, page=page, seed=72).fill()
    _check_nan_attention(_with_nans(s, [(0, 385, "k", 0, 1), (0, 388, "k", 1, 2), (1, 70, "k", 0, 9), (1, 66, "k", 1, 0),
                                        (2, 202, "k", 0, 5), (2, 201, "k", 1, 6)]), torch.bfloat16, G)


@pytest.mark.parametrize("D,page,G", [(128, 64, 1), (64, 16, 4), (128, 32, 2)])
def test_nan_values_that_every_row_sees(D, page, G):
    """NaN values of cached tokens, in whole steps and in an incomplete one (all the keys of sequence 1)."""
    s = Setup([90, 70, 1], [300, 20, 200], H=2, D=D, page=page, seed=73).fill()
    _check_nan_attention(_with_nans(s, [(0, 7, "v", 0, 1), (1, 3, "v", 1, 60), (1, 3, "v", 1, 61), (2, 199, "v", 0, 5)]),
                         torch.float16, G)
    s = Setup([90, 70], [300, 20], H=2, D=D, page=page, seed=74).fill()
    _check_nan_attention(_with_nans(s, [(0, 389, "v", 0, 1), (1, 88, "v", 1, 60)]), torch.bfloat16, G, causal=False)


@pytest.mark.parametrize("new,ctx,G,longest", [
    ([3, 2, 1], [100, 700, 30], 4, None),        # a few new tokens each
    ([4, 2, 1], [100, 700, 30], 4, 200000),      # in chunks
    ([90, 300, 65], [300, 5, 0], 1, None),       # prompts
    ([120], [3000], 2, None)])                   # a prompt in chunks
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
def test_nan_values_behind_a_row(new, ctx, G, longest, D, page):
    """NaN values of the new tokens themselves: they reach the rows that see them, in their elements
    only, and no row before them."""
    s = Setup(new, ctx, H=2, D=D, page=page, seed=75, width=-(-(longest or 4000) // page)).fill()
    at = []
    for b, n in enumerate(s.new):
        for back, h, d in ((1, 0, 0), (2, 1, 7), (n // 2 + 1, 0, D - 1), (n // 2 + 1, 0, 0), (n - 1, 1, 33)):
            if 0 < back <= n:
                at.append((b, s.lens[b] - back, "v", h, d))
    _check_nan_attention(_with_nans(s, at), torch.bfloat16, G, max_seq_len=longest)


# ------------------------------------------------------------------------------------
# pages far apart in size
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,ctx,G", [([2], [200], 4), ([100], [200], 1), ([90], [1500], 2)])
def test_values_of_pages_far_apart(page, D, new, ctx, G):
    """Pages of values 2^45 to 2^75 larger than those that carry the probability: before them, beside
    them in the same step, and behind them, where some rows do not see them. The large pages' keys have
    a score 25600 below the others' at least, so their probability is zero and the tolerance is that of
    the others alone: their probabilities are equal, so nothing but roundings of 2^-11 and the sums."""
    s = Setup(new, ctx, H=1, D=D, page=page, seed=80).fill()
    pages = s.table[0, :-(-s.lens[0] // page)]
    plus, minus = (osv.e4m3_encode(np.full((page, D), x)) for x in (100.0, -100.0))
    for i, pg in enumerate(pages):
        large = i % 4 == 2 or i == len(pages) - 1
        s.k[pg, 0], s.ks[pg, 0] = (minus if large else plus), 127
        s.v[pg, 0] = osv.e4m3_encode(s.rng.standard_normal((page, D)) * 50)
        s.vs[pg, 0] = 127 + (30 + i % 10 if large else -36 + i % 22)
    q = torch.full((new[0], G, D), 2.0, dtype=torch.bfloat16, device="cuda")
    out, lse = s.cache().attention(q, *s.batch(), max_q_len=new[0], scale=1.0, return_lse=True)
    ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 1.0, True)
    assert np.abs(ro).max() < 100 and info["vmax"].max() > 2.0 ** 30
    tol = (2.0 ** -10 + (s.lens[0] + 66) * 2.0 ** -23) * info["pv"] + 2.0 ** -8 * np.abs(ro)
    assert np.all(np.abs(f64(out) - ro) <= tol)
    assert np.all(np.abs(f64(lse) - rl) <= 2.0 ** -18 + 2.0 ** -22 * np.abs(rl))


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("new,ctx,G", [([2], [200], 4), ([100], [200], 1), ([90], [1500], 2)])
def test_keys_of_pages_far_apart(page, new, ctx, G):
    """Keys of 2^-30 to 2^-14 that carry the probability beside keys of 2^10 and more whose scores are
    hugely negative: the small keys' scores differ and have to keep their bits."""
    D = 64
    s = Setup(new, ctx, H=1, D=D, page=page, seed=81).fill()
    pages = s.table[0, :-(-s.lens[0] // page)]
    small = np.zeros(len(pages) * page, dtype=bool)
    for i, pg in enumerate(pages):
        large = i % 4 == 2 or i == len(pages) - 1
        small[i * page:(i + 1) * page] = not large
        x = s.rng.standard_normal((page, D)) * 100
        s.k[pg, 0] = osv.e4m3_encode(-np.abs(x) if large else x)
        s.ks[pg, 0] = 127 + (6 + i % 20 if large else -30 + i % 8)
    small = small[:s.lens[0]]
    rng = np.random.default_rng(1)
    q = torch.from_numpy(2.0 ** 20 * (1 + rng.random((new[0], G, D)))).to(torch.bfloat16).cuda()  # positive
    scale = 2.0 ** -3
    out, lse = s.cache().attention(q, *s.batch(), max_q_len=new[0], scale=scale, return_lse=True)
    ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, scale, True)
    k = osv.kv_values(s.k, s.ks, s.table[0], s.lens[0])[:, 0]
    z = scale * np.einsum("tgd,jd->tgj", f64(q), k)
    assert z[:, :, ~small].max() < -2.0 ** 20 and 0.5 < z[:, :, small].max() < 100  # and they do differ
    a = scale * np.einsum("tgd,jd->tgj", np.abs(f64(q)), np.abs(k[small])).max()
    e = (D * 2.0 ** -23 + 2.0 ** -21) * a
    n = s.lens[0]
    assert np.all(np.abs(f64(lse) - rl) <= e + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(rl)))
    tol = (2 * e + 2.0 ** -11 + (n + 66) * 2.0 ** -23) * info["pv"] + n * 2.0 ** -25 * info["vmax"][..., None]
    assert np.all(np.abs(f64(out) - ro) <= tol + 2.0 ** -8 * np.abs(ro))


def test_units_of_pages_change_often():
    """Pages of every size of the whole range, in steps of 16 and of 128 keys: each row against the
    largest product of probability and value that it sees (the sums are float32)."""
    for page, D in ((16, 64), (128, 128), (32, 128)):
        s = Setup([150, 70], [900, 0], H=2, D=D, page=page, seed=82).fill()
        s.vs[:] = 127 + s.rng.integers(-40, 41, s.vs.shape)
        s.ks[:] = np.minimum(s.ks, 122) - s.rng.integers(0, 30, s.ks.shape)
        q = torch.randn(220, 2, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
        cache = s.cache()
        out, lse = cache.attention(q, *s.batch(), max_q_len=150, scale=0.125, return_lse=True)
        assert cache.device_status() == 0
        ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 0.125, True)
        n = max(s.lens)
        e = ((D * 2.0 ** -23 + 2.0 ** -21) * info["a"])[..., None]
        tol = (2 * e + 2.0 ** -11 + (n + 66) * 2.0 ** -23) * info["pv"] + n * 2.0 ** -25 * info["vmax"][..., None]
        assert np.all(np.abs(f64(out) - ro) <= tol + 2.0 ** -8 * np.abs(ro))


# ------------------------------------------------------------------------------------
# probabilities far below the largest
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("new,ctx,G,longest", [
    ([1], [3000], 4, None), ([1], [3000], 4, 60000), ([3], [200], 2, None),  # one chunk, a cluster's, the workspace's
    ([100], [3000], 1, None), ([300], [20], 2, None)])                       # prompts
@pytest.mark.parametrize("gap", [16, 24])
def test_a_dominating_key_without_value(new, ctx, G, longest, gap):
    """One key holds all but a few millionths of the probability and its value is zero: the output is the
    others'. With a gap of 16 +- 1 (2^-24.6) every probability is rounded by 2^-11, so the tolerance is
    relative to the others; with 24 (2^-36.1) 2^-37 of the largest is added."""
    D, page = 64, 64
    s = Setup(new, ctx, H=1, D=D, page=page, seed=90, width=-(-(longest or 4000) // page)).fill()
    pages = s.table[0, :-(-s.lens[0] // page)]
    for pg in pages:
        s.k[pg, 0] = osv.e4m3_encode(s.rng.uniform(-1.0, 1.0, (page, D)) / 32)  # scores of at most 1 beside q = 1
        s.v[pg, 0] = osv.e4m3_encode(1.0 + s.rng.uniform(0.0, 1.0, (page, D)))
        s.ks[pg, 0] = s.vs[pg, 0] = 127
    s.k[pages[0], 0, 0], s.v[pages[0], 0, 0] = osv.e4m3_encode(np.full(D, gap / D)), 0
    n = new[0]
    q = torch.full((n, G, D), 0.5, dtype=torch.bfloat16, device="cuda")
    out, lse = s.cache().attention(q, *s.batch(), max_q_len=n, max_seq_len=longest or s.lens[0], scale=2.0, return_lse=True)
    ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 2.0, True)
    e = ((D * 2.0 ** -23 + 2.0 ** -21) * info["a"])[..., None]
    tol = (2 * e + 2.0 ** -11 + (s.lens[0] + 66) * 2.0 ** -23) * info["pv"] + 2.0 ** -8 * np.abs(ro)
    if gap > 17:
        tol += s.lens[0] * 2.0 ** -37 * info["vmax"][..., None]
    assert 0 < np.abs(ro).max() < 2.0 ** -10
    assert np.all(np.abs(f64(out) - ro) <= tol), float((np.abs(f64(out) - ro) / tol).max())
    assert np.all(np.abs(f64(lse) - rl) <= e[..., 0] + (s.lens[0] + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(rl)))


# ------------------------------------------------------------------------------------
# bounds of a call that its batch passes
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("new,ctx,G,bound", [
    ([100], [30], 1, 64), ([100, 3, 90], [30, 200, 0], 1, 64),  # the call's rows fit the one kernel, the sequences' do not
    ([300, 20], [10, 700], 2, 130), ([300], [2000], 1, 80),     # prompts, whole and in chunks
    ([20, 3], [600, 2500], 4, 1), ([20, 3], [600, 2500], 4, 2), ([9], [40], 3, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_more_new_tokens_than_max_q_len(new, ctx, G, bound, causal):
    """The first max_q_len queries of a longer sequence are computed, the others' rows are not written,
    and the batch is reported."""
    s = Setup(new, ctx, H=2, D=64, page=32, seed=91).fill()
    n, Hq = s.cu[-1], 2 * G
    q = torch.randn(n, Hq, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    cache = s.cache()
    out = torch.full((n, Hq, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, Hq), 9.0, device="cuda")
    cache.attention(q, *s.batch(), max_q_len=bound, max_seq_len=max(s.lens), causal=causal, out=out, lse=lse, return_lse=True)
    assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
    index = np.concatenate([np.arange(c) for c in new])
    done, left = index < bound, torch.from_numpy(index >= bound).cuda()
    assert bool((out[left] == 9.0).all()) and bool((lse[left] == 9.0).all())
    ro, rl, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 0.125, causal)
    keys = max(s.lens)
    e = (64 * 2.0 ** -23 + 2.0 ** -21) * info["a"]
    tol = ((2 * e + 2.0 ** -11 + (keys + 66) * 2.0 ** -23)[..., None] * info["pv"]
           + keys * 2.0 ** -25 * info["vmax"][..., None] + 2.0 ** -8 * np.abs(ro))
    assert np.all((np.abs(f64(out) - ro) <= tol)[done])
    ltol = e + (keys + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(rl))
    assert np.all((np.abs(f64(lse) - rl) <= ltol)[done])


@pytest.mark.parametrize("cu,lens", [
    ([0, 3, 1, 5], [9, 9, 9]),         # fewer new tokens than none
    ([0, 5, 5, 4], [9, 9, 9]), ([0, 2, 2, 7], [9, 9, 9]), ([40, 41, 41, 41], [9, 9, 9]), ([0, 2, 2, 2000000000], [9, 9, 9]),
    ([-3, -2, 0, 5], [9, 9, 9]), ([0, 2, 5, 5], [9, 2, 9]), ([0, 2, 2, 5], [9, -1, 9])])
def test_batches_out_of_range_are_reported(cu, lens):
    """Both calls report a batch whose rows fall, end behind the arrays or begin there, or whose lengths
    are shorter than the new tokens."""
    cache = KVCache(6, 16, 1, 64)
    x = torch.randn(5, 1, 64, device="cuda").half()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[0], [1], [2]])
    cache.append(x, x, i32(cu), i32(lens), table, q=x, inv_freq=torch.ones(16, device="cuda"))
    assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
    cache.attention(x, i32(cu), i32(lens), table, max_q_len=5)
    assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
    cache.append(x, x, i32([0, 2, 2, 5]), i32([2, 0, 4]), table)
    cache.attention(x, i32([0, 2, 2, 5]), i32([2, 0, 4]), table, max_q_len=3)
    assert cache.device_status() == 0


# ------------------------------------------------------------------------------------
# streams and threads
# ------------------------------------------------------------------------------------
def test_device_status_covers_other_streams():
    """A bad batch queued on another stream behind a delay is reported, once."""
    cache = KVCache(4, 16, 1, 64)
    x = torch.randn(2, 1, 64, device="cuda").half()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cu, good, bad, table, out = i32([0, 2]), i32([2]), i32([1]), i32([[0]]), torch.empty_like(x)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda n: cache.append(x, x, cu, n, table, stream=st),
                 lambda n: cache.attention(x, cu, n, table, 2, out=out, stream=st)):
        call(good)  # (the first call loads the kernel, which waits for the device)
        assert cache.device_status() == 0
        with torch.cuda.stream(st):
            torch.cuda._sleep(40_000_000)  # about 20 ms
        call(bad)
        assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
        call(good)
        assert cache.device_status() == 0


def test_memory_of_the_given_stream_in_every_mode():
    """Outputs of the per-group calls and of the rotation alone, too, come from the given stream's memory:
    not what the current stream has freed but still has to read."""
    K, M, N = 32, 16, 16
    x = torch.randn(K, M, N, device="cuda").to(torch.bfloat16)
    eye = torch.eye(16, device="cuda").to(torch.bfloat16)
    fq, st = FlatQuant(K, M, N), torch.cuda.Stream()
    for call in (lambda: fq.quantize_mx(x, eye, eye, stream=st), lambda: quantize_mx_static(x, eye, eye, stream=st),
                 lambda: (fq.debug_rotate(x, eye, eye, stream=st),),
                 lambda: fq.quantize_per_token(x, eye, eye, stream=st),
                 lambda: fq.quantize_per_token(x, eye, eye, out_dtype="int32", stream=st)):
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (8, 256, 1024, 4096, 16384, 65536)
                for _ in range(64)]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # about 20 ms
        copies = [h.clone() for h in held]
        del held  # free, and read by the copies that are still queued
        got = call()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bounds_given_as_tensors_that_change():
    """max_seq_len as a host tensor that a server counts up in place: the workspace follows its value."""
    s = Setup([1], [9000], H=1, D=64, page=64, seed=92, width=400).fill()
    cache, batch = s.cache(), s.batch()
    q = torch.randn(1, 2, 64, device="cuda").half()
    longest = torch.tensor(1000)
    short = (batch[0], torch.tensor([900], dtype=torch.int32, device="cuda"), batch[2])
    cache.attention(q, *short, max_q_len=1, max_seq_len=longest)
    longest.fill_(25000)
    got = cache.attention(q, *batch, max_q_len=1, max_seq_len=longest)
    assert torch.equal(got, cache.attention(q, *batch, max_q_len=1, max_seq_len=25000)) and cache.device_status() == 0


@pytest.mark.parametrize("new,ctx,G,longest", [([1], [900], 4, None), ([1], [900], 4, 60000), ([3], [200], 2, None),
                                               ([100], [900], 1, None), ([300], [20], 2, None)])
@pytest.mark.parametrize("size", [2.0 ** 18, 2.0 ** 24, 2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_past_the_exponents_range(new, ctx, G, longest, size, sign):
    """Scores of 10^5 to 10^20: one key takes all of a row's probability, the output is its value (the
    values' own half step aside) and lse its score, by the score's float32 roundings."""
    D = 128
    s = Setup(new, ctx, H=1, D=D, page=64, seed=93, width=-(-(longest or 1000) // 64)).fill()
    n = new[0]
    q = torch.randn(n, G, D, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    scale = sign * size
    out, lse = s.cache().attention(q.cuda(), *s.batch(), max_q_len=n, max_seq_len=longest or s.lens[0], scale=scale,
                                   return_lse=True)
    k, v = (osv.kv_values(c, x, s.table[0], s.lens[0])[:, 0] for c, x in ((s.k, s.ks), (s.v, s.vs)))
    z = scale * np.einsum("tgd,jd->tgj", f64(q), k)
    seen = s.lens[0] - n + np.arange(n) + 1
    z[np.broadcast_to(np.arange(s.lens[0]) >= seen[:, None, None], z.shape)] = -np.inf
    at, err = z.argmax(-1), (D * 2.0 ** -23 + 2.0 ** -21) * size * (np.abs(f64(q)) @ np.abs(k).max(0))
    second = np.sort(z, -1)[..., -2]
    clear = z.max(-1) - second > 2 * err + 60  # the others are below 2^-86
    assert clear.mean() > 0.9
    assert np.all(np.isfinite(f64(out))) and np.all(np.isfinite(f64(lse)))
    assert np.all(np.abs(f64(out) - v[at])[clear] <= 2.0 ** -8 * np.abs(v[at])[clear])
    assert np.all(np.abs(f64(lse) - z.max(-1))[clear] <= (err + 2.0 ** -22 * np.abs(z.max(-1)))[clear])


def test_two_threads_on_one_cache():
    """Two threads with a stream each call append and attention on one cache, on pages and sizes of their own."""
    cache = KVCache(64, 16, 2, 64)
    sizes = ((1, 300), (40, 200))

    def inputs(i):
        n, ctx = sizes[i]
        g = torch.Generator(device="cuda").manual_seed(i)
        total = n + ctx
        table = torch.arange(32 * i, 32 * i + 32, dtype=torch.int32, device="cuda")[None]
        k, v = (torch.randn(total, 2, 64, generator=g, device="cuda").half() for _ in range(2))
        q = torch.randn(n, 8, 64, generator=g, device="cuda").half()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return k, v, q, i32([0, total]), i32([0, n]), i32([total]), table, n, total

    def run(c, k, v, q, cu_all, cu, lens, table, n, total, reps):
        outs = []
        for _ in range(reps):
            c.append(k, v, cu_all, lens, table)
            outs.append(c.attention(q, cu, lens, table, max_q_len=n, max_seq_len=total))
        return outs

    data = [inputs(i) for i in range(2)]
    want = [run(KVCache(64, 16, 2, 64), *d, reps=1)[0] for d in data]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got[i] = run(cache, *data[i], reps=50)
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert cache.device_status() == 0
    for i in range(2):
        assert len(got[i]) == 50 and all(torch.equal(o, want[i]) for o in got[i])


# ------------------------------------------------------------------------------------
# many sequences, and prompts beside decode steps
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("count", [33, 65, 1100])
def test_append_many_sequences(count):
    """More sequences than a warp probes at once, and than two rounds of probes tell apart; some without
    new tokens."""
    r = np.random.default_rng(count)
    new = r.integers(0, 4, count).tolist()
    s = Setup(new, r.integers(0, 40, count).tolist(), H=1, D=64, page=16, seed=94)
    _check_append(s, torch.bfloat16, G=2, rot=32, interleaved=False, tail=3)


def test_prompts_of_many_sequences():
    """More sequences than the prompt kernel sorts by length."""
    r = np.random.default_rng(1)
    s = Setup([9] * 259 + [1, 0, 20], r.integers(0, 40, 262).tolist(), H=1, D=64, page=16, seed=95).fill()
    _check_attention(s, torch.bfloat16, G=8)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 1)])
def test_prompts_beside_decode_steps(D, G):
    """Prompts, whole and in chunks, and decode steps whose contexts are divided into more chunks than a
    cluster joins, in one call."""
    s = Setup([200, 1, 1, 130, 3, 0, 1], [0, 9000, 40, 700, 6000, 10, 3000], H=1, D=D, page=64, seed=96).fill()
    _check_attention(s, torch.bfloat16, G=G, tail=2)
    _check_attention(s, torch.float16, G=G, causal=False)


def test_host_pipeline_int8():
    """INT8 codes from host memory in slices: those of one call on the device."""
    K, M, N = 64, 64, 64
    g = torch.Generator().manual_seed(8)
    x = torch.randn(K, M, N, generator=g).to(torch.bfloat16)
    P1, P2 = (torch.linalg.qr(torch.randn(n, n, generator=g))[0].to(torch.bfloat16).contiguous() for n in (M, N))
    fq = FlatQuant(K, M, N)
    want = fq.quantize_per_token(x.cuda(), P1.cuda(), P2.cuda(), out_dtype="int8")
    for chunks in (1, 4):
        pipe = HostPipeline(fq, "per_token", out_dtype="int8", chunks=chunks)
        out, scale = pipe.host_outputs()
        pipe.run(x.pin_memory(), P1.pin_memory(), P2.pin_memory(), out, scale)
        torch.cuda.synchronize()
        assert out.dtype is torch.int8 and torch.equal(out, want[0].cpu()) and torch.equal(scale, want[1].cpu())


@pytest.mark.parametrize("new,ctx", [([6], [70]), ([100], [70])])
def test_queries_up_to_the_largest_and_down_to_the_smallest(new, ctx):
    """Rows of q up to 2^127 and down to 2^-126 with scores scaled back: the same result."""
    s = Setup(new, ctx, H=1, D=128, page=32, seed=97).fill()
    base = torch.randint(1, 4, (new[0], 1, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16) * 0.25
    cache = s.cache()
    call = lambda e: cache.attention((base * 2.0 ** e).cuda(), *s.batch(), max_q_len=new[0], scale=0.1 * 2.0 ** -e)  # noqa: E731
    want = call(0)
    ro, _, info = osv.kv_attention(f64(base), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 0.1, True)
    assert np.all(np.abs(f64(want) - ro) <= (2.0 ** -8 + 2.0 ** -10) * info["pv"] + 2.0 ** -17 * info["vmax"][..., None])
    for e in (98, -98):  # (the scale is at most 1e30)
        assert torch.equal(call(e), want)
    # with scores that stay large or small: finite, the largest score's value or the mean
    for e in (115, 127):
        out, lse = cache.attention((base * 2.0 ** e).cuda(), *s.batch(), max_q_len=new[0], scale=2.0 ** -99, return_lse=True)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        ro, rl, info = osv.kv_attention(f64(base) * 2.0 ** e, s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 2.0 ** -99, True)
        err = (128 * 2.0 ** -23 + 2.0 ** -21) * info["a"]
        assert np.all(np.abs(f64(lse) - rl) <= err + 2.0 ** -13 + 2.0 ** -22 * np.abs(rl))


def test_prompt_past_four_gigabytes():
    """A prompt's pages whose codes lie past 2^32 bytes."""
    H, D, page, n = 8, 128, 128, 100
    pages = (1 << 32) // (H * D * page) + 40
    cache = KVCache(pages, page, H, D)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, total = i32([[pages - 1, 7, pages - 3]]), 2 * page + 9
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(total, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.append(k, v, i32([0, total]), i32([total]), table)
    q = torch.randn(n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = cache.attention(q, i32([0, n]), i32([total]), table, max_q_len=n)
    small = KVCache(3, page, H, D)
    small.append(k, v, i32([0, total]), i32([total]), i32([[0, 1, 2]]))
    want = small.attention(q, i32([0, n]), i32([total]), i32([[0, 1, 2]]), max_q_len=n)
    assert cache.device_status() == 0 and torch.equal(out, want)


# ------------------------------------------------------------------------------------
# INT8 codes
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("kernel,K,M,N", [("general", 5, 16, 16), ("general", 4, 7, 33), ("tcgen05", 40, 64, 64),
                                          ("tcgen05", 20, 128, 112)])
@pytest.mark.parametrize("exponent", [-112, -122, -125])
def test_int8_codes_of_tiny_tokens(kernel, K, M, N, exponent):
    """Tokens of 2^exponent, whose quantScale's reciprocal is past float32 (the scale below 2^-128, the last two). With
    identity rotations x'' = x and a code is x / quantScale: within half, the scale's own rounding (half a step,
    2^-150 at the bottom of the range) and the product's two roundings aside."""
    g = np.random.default_rng([K, M, N])
    x = torch.from_numpy((g.integers(-128, 129, (K, M * N)) / 128.0).astype(np.float32)).to(torch.bfloat16) * 2.0 ** exponent
    x[:, 0] = 2.0 ** exponent
    x[1] = 0.0
    eye = [torch.eye(n, dtype=torch.bfloat16, device="cuda") for n in (M, N)]
    codes, qs = FlatQuant(K, M, N, kernel=kernel).quantize_per_token(x.view(K, M, N).cuda(), *eye, out_dtype="int8")
    s = 2.0 ** exponent / 127
    want = np.full(K, s)
    want[1] = 0.0
    assert np.all(np.abs(f64(qs) - want) <= 2.0 ** -24 * s + 2.0 ** -150)
    v = f64(x) / s
    rel = 2.0 ** -22 + 2.0 ** -150 / s
    off = np.abs(codes.cpu().numpy().astype(np.float64) - v)
    assert np.all(off <= 0.5 + np.abs(v) * rel), float(off.max())
