"""GPU tests of the 8-bit paged cache: KVCache.append and KVCache.attention against the float64
oracle (`oracle/serving.py`), and a run of the whole path.

Tolerances, derived from the arithmetic:
* values of v are stored by one rounding: codes and bytes equal the oracle's.
* rotated values: sin and cos are off by at most 2^-22 (the reduced angle as float32 and the
  function itself) and the two products and their sum by 2^-24 each, so |dx| <= 2^-21 (|x| + |y|)
  for the pair (x, y); q then by half a step of its type. A code of k differs from the oracle's
  only where that moves it over a rounding border; compared by value: half a step of E4M3 (2^-4
  relative, or 2^-10 units below the normal range) beside dx. The page's byte may differ only
  where the maximum lies within dx of 448 * 2^e.
* attention: a score's float32 sum over D exact products and its scaling are off by
  e = (D 2^-23 + 2^-21) a, a = max_j scale sum_d |q_d k_jd| (and 2^-38 of it for q's conversion); a
  probability by 2 e + 2^-22 + 2^-11 relative (its rounding to fp16, an absolute 2^-25 at the bottom
  of the range), the sums over n keys and the rescalings by (n + 64) 2^-23 relative. So
  |do| <= (2 e + 2^-11 + (n + 66) 2^-23) sum_j p_j |v_j| + n 2^-25 max|v| + half a step of o, and
  |dlse| <= e + (n + 64) 2^-23 + 2^-22 (1 + |lse|).
"""

import numpy as np
import pytest
import torch

from oracle import serving as osv
from rotation_bit_quantization_token_b200 import FQError, FlatQuant, KVCache, _lib, int8_matmul

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
f64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A cache in use and a batch of sequences with `new` tokens on top of `ctx` cached ones."""

    def __init__(self, new, ctx, H=2, D=128, page=32, seed=0, spare=3, width=None):
        self.rng = np.random.default_rng([seed, H, D, page, len(new)])
        self.new, self.lens = list(new), [n + c for n, c in zip(new, ctx)]
        self.cu = [0] + np.cumsum(new).tolist()
        self.H, self.D, self.page = H, D, page
        need = [-(-n // page) for n in self.lens]
        self.pages = sum(need) + spare
        order = self.rng.permutation(self.pages)
        self.width = width or max(need + [1])
        self.table = np.full((len(new), self.width), -1, dtype=np.int32)  # unused entries are not pages
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, H, page, D)
        # contents: finite codes of all sizes in tokens that exist, NaN codes everywhere else
        self.k, self.v = (np.full(shape, 0x7F, dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full(shape[:2], 127, dtype=np.uint8) for _ in range(2))
        for b, c in enumerate(ctx):
            for p in range(-(-c // page)):
                rows = min(page, c - p * page)
                for codes, sc, lo, hi in ((self.k, self.ks, -4, 0), (self.v, self.vs, -14, 3)):
                    for h in range(H):
                        x = self.rng.standard_normal((rows, D)) * 2.0 ** self.rng.integers(lo, hi)
                        e = osv.page_exponent(np.abs(x).max())
                        codes[self.table[b, p], h, :rows] = osv.e4m3_encode(x * 2.0 ** -e)
                        sc[self.table[b, p], h] = e + 127

    def fill(self):
        """The new tokens' rows too (for attention alone)."""
        new = [self.rng.standard_normal((self.cu[-1], self.H, self.D)) * s for s in (1.0, 1.5)]
        osv.kv_store(self.k, self.ks, new[0], self.cu, self.lens, self.table)
        osv.kv_store(self.v, self.vs, new[1], self.cu, self.lens, self.table)
        return self

    def cache(self):
        t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        return KVCache.from_buffers(t(self.k).view(torch.float8_e4m3fn), t(self.v).view(torch.float8_e4m3fn),
                                    t(self.ks), t(self.vs))

    def batch(self):
        return _i32(self.cu), _i32(self.lens), torch.from_numpy(self.table).cuda()


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------
def _check_append(s, dtype, G, rot, interleaved, tail=0, strided=True, gain=1.0):
    T = s.cu[-1] + tail
    g = torch.Generator().manual_seed(1)
    Hq = s.H * G
    qkv = torch.randn(T, Hq + 2 * s.H, s.D, generator=g) * torch.exp(torch.randn(T, Hq + 2 * s.H, 1, generator=g)) * gain
    qkv = qkv.to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + s.H], qkv[:, Hq + s.H:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    f = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda() if rot else None
    cache = s.cache()
    q_out = torch.full((T, Hq, s.D), 7.0, dtype=dtype, device="cuda")
    got = cache.append(k, v, *s.batch(), q=q, inv_freq=f, interleaved=interleaved, q_out=q_out)
    assert got is q_out and cache.device_status() == 0
    # the oracle
    n = s.cu[-1]
    pos = np.concatenate([np.arange(L - c, L) for c, L in zip(s.new, s.lens)])
    fr = f64(f) if rot else np.zeros(0)
    wq, wk = osv.rotary(f64(q[:n]), pos, fr, interleaved), osv.rotary(f64(k[:n]), pos, fr, interleaved)

    def pair(x):  # |x| + |partner| of every element
        y = np.abs(x).copy()
        h = rot // 2
        i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), np.arange(h) + h)
        z = y[..., i0] + y[..., i1]
        y[..., i0], y[..., i1] = z, z
        y[..., rot:] = 0.0
        return y

    dq = 2.0 ** -21 * pair(f64(q[:n]))
    tiny = 2.0 ** -25 if dtype is torch.float16 else 0.0
    assert np.all(np.abs(f64(q_out[:n]) - wq) <= dq + HALF[dtype] * (np.abs(wq) + dq) + tiny)
    assert torch.all(q_out[n:] == 7.0)  # rows behind the last sequence
    rk, rks, rv, rvs = s.k.copy(), s.ks.copy(), s.v.copy(), s.vs.copy()
    osv.kv_store(rk, rks, wk, s.cu, s.lens, s.table)
    osv.kv_store(rv, rvs, f64(v[:n]), s.cu, s.lens, s.table)
    assert np.array_equal(cache.v_scale.cpu().numpy(), rvs)
    assert np.array_equal(_codes(cache.v), rv)  # new rows, re-rounded older rows, untouched others
    gk, gks = _codes(cache.k), cache.k_scale.cpu().numpy()
    if not rot:
        assert np.array_equal(gk, rk) and np.array_equal(gks, rks)
        return cache
    dk = 2.0 ** -21 * pair(f64(k[:n]))
    assert np.mean(gks != rks) <= 0.01 and np.all(np.abs(gks.astype(int) - rks) <= 1)
    for b in range(len(s.new)):
        for i in range(s.new[b]):
            at = s.lens[b] - s.new[b] + i
            pg, r, t = s.table[b, at // s.page], at % s.page, s.cu[b] + i
            unit = np.exp2(gks[pg].astype(float) - 127)[:, None]
            val = osv.E4M3[gk[pg, :, r]] * unit
            lim = np.maximum(2.0 ** -4 * np.abs(wk[t]), 2.0 ** -10 * unit) + dk[t] * (1 + 2.0 ** -4)
            # a maximum within dk of 448 * 2^e may saturate
            lim = np.where(np.abs(wk[t]) > 448 * unit, np.maximum(lim, np.abs(wk[t]) - 448 * unit), lim)
            assert np.all(np.abs(val - wk[t]) <= lim), (b, i)
            gk[pg, :, r] = rk[pg, :, r] = 0
    same = gks == rks
    assert np.array_equal(gk[same], rk[same])  # older rows and untouched ones
    return cache


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_decode_steps(page, D, dtype):
    """One new token each: first of a sequence, first of a page, inside a page, last of a page,
    and sequences without new tokens."""
    s = Setup([1, 1, 1, 0, 1, 1], [0, page, page - 1, 9, 5, 2 * page + 3], D=D, page=page)
    _check_append(s, dtype, G=3, rot=D, interleaved=False)


@pytest.mark.parametrize("page,D,rot,il", [(16, 128, 128, True), (32, 64, 32, False), (64, 128, 64, True), (128, 64, 64, False),
                                           (128, 128, 0, False), (16, 64, 16, True), (64, 64, 48, False)])
def test_append_prompts(page, D, rot, il):
    """Prompts over many pages, from the middle of a page, with a tail of unused rows."""
    s = Setup([70, 1, 300, 17], [0, 200, 37, page - 1], H=3, D=D, page=page, seed=2)
    _check_append(s, torch.bfloat16, G=2, rot=rot, interleaved=il, tail=5)


def test_append_grows_and_keeps_exponents():
    """New tokens far above and far below the page's older ones: the older codes move to the new
    exponent (subnormal results rounded once, far ones to zero), or the page keeps its own."""
    for gain in (2.0 ** 6, 2.0 ** 14, 2.0 ** -9, 2.0 ** -20):
        s = Setup([3, 1, 20], [5, 40, 30], H=2, D=128, page=64, seed=3)
        _check_append(s, torch.bfloat16, G=1, rot=0, interleaved=False, strided=False, gain=gain)


def test_append_extreme_magnitudes():
    """Zeros, the smallest and largest numbers of the type, infinities: bytes stay in [87, 167] and
    codes finite."""
    s = Setup([4, 3], [0, 2], H=1, D=64, page=16)
    cache = s.cache()
    k = torch.zeros(7, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[1, 0, 5], k[2, 0, 0], k[4, 0, 3], k[5, 0, 1] = 1e-38, -3e38, float("inf"), 1.0
    v = torch.zeros_like(k)
    cache.append(k, v, *s.batch())
    ks, vs = cache.k_scale.cpu().numpy(), cache.v_scale.cpu().numpy()
    assert ks[s.table[0, 0], 0] == 167 and ks[s.table[1, 0], 0] == 167
    assert vs[s.table[0, 0], 0] == 87
    ck = _codes(cache.k)[s.table[0, 0], 0]
    assert ck[2, 0] == 0xFE and np.all(ck[:4, 1:] == 0) and _codes(cache.k)[s.table[1, 0], 0, 2, 3] == 0x7E
    assert np.all(_codes(cache.v)[s.table[0, 0], 0, :4] == 0)


def test_append_far_positions():
    """Positions near 10^6: the angle needs more than float32 (its rounding alone would be 0.06)."""
    page, n = 128, 1_000_003
    width = n // page + 1
    s = Setup([2], [0], H=1, D=64, page=page, width=width)
    s.table[0, :] = -1
    s.table[0, (n - 2) // page], s.table[0, (n - 1) // page] = 0, 0
    f = torch.full((32,), 0.7310585, device="cuda")
    q = torch.zeros(2, 1, 64, dtype=torch.float16, device="cuda")
    q[:, :, :32] = 1.0
    cache = s.cache()
    cu, _, table = s.batch()
    out = cache.append(q, q, cu, _i32([n]), table, q=q, inv_freq=f)
    ang = (n - 2 + np.arange(2.0)) * float(f[0])
    assert np.all(np.abs(f64(out)[:, 0, 0] - np.cos(ang)) <= 2.0 ** -21 + 2.0 ** -11)
    assert np.all(np.abs(f64(out)[:, 0, 32] - np.sin(ang)) <= 2.0 ** -21 + 2.0 ** -11)


def test_append_is_repeatable():
    s = Setup([40, 1, 3], [10, 64, 100], page=64, seed=5)
    runs = []
    for _ in range(2):
        cache = _check_append(s, torch.float16, G=2, rot=64, interleaved=False)
        runs.append([_codes(cache.k), _codes(cache.v), cache.k_scale.cpu().numpy()])
    assert all(np.array_equal(a, b) for a, b in zip(*runs))


def test_append_bad_batches_are_refused():
    """Contents that are out of range store nothing where they are wrong, and are reported."""
    def run(change, expect=_lib.FQ_KV_BAD_BATCH):
        s = Setup([2, 3], [1, 20], H=2, D=64, page=16, seed=6)
        cu, lens, table = (x.cpu().clone() for x in s.batch())
        change(cu, lens, table)
        cache = s.cache()
        k = torch.randn(5, 2, 64, device="cuda").half()
        cache.append(k, k, cu.cuda(), lens.cuda(), table.cuda())
        assert cache.device_status() == expect
        assert cache.device_status() == 0
        return s, _codes(cache.k)

    def untouched(s, k, b):
        pages = [p for p in s.table[b] if p >= 0]
        return np.array_equal(k[pages], s.k[pages])

    for page in (-1, 10 ** 6, -(2 ** 31), 2 ** 31 - 1):
        s, k = run(lambda cu, lens, table: table.__setitem__((1, 1), page))
        assert untouched(s, k, 1) and not untouched(s, k, 0)
    s, k = run(lambda cu, lens, table: lens.__setitem__(0, 1))         # two new tokens, length 1
    assert untouched(s, k, 0) and not untouched(s, k, 1)
    s, k = run(lambda cu, lens, table: lens.__setitem__(1, 2 ** 31 - 1))  # past the table
    assert untouched(s, k, 1)
    s, k = run(lambda cu, lens, table: cu.__setitem__(2, 2000))        # rows past T
    assert untouched(s, k, 1) and not untouched(s, k, 0)
    s, k = run(lambda cu, lens, table: cu.__setitem__(0, -7))
    assert untouched(s, k, 0)
    s, k = run(lambda cu, lens, table: None, expect=0)
    assert not untouched(s, k, 0) and not untouched(s, k, 1)


# ------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------
def _check_attention(s, dtype, G, causal=True, scale=None, gain=2.0, tail=0, max_seq_len=None, cache=None, strided=False):
    Hq, D, n = s.H * G, s.D, s.cu[-1]
    g = torch.Generator().manual_seed(9)
    q = (gain * torch.randn(n + tail, Hq + (2 if strided else 0), D, generator=g)).to(dtype).cuda()[:, :Hq]
    scale = D ** -0.5 if scale is None else scale
    cache = cache or s.cache()
    out = torch.full((n + tail, Hq, D), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((n + tail, Hq), 9.0, device="cuda")
    got = cache.attention(q, *s.batch(), max_q_len=max(s.new), max_seq_len=max_seq_len or max(s.lens + [1]), scale=scale,
                          causal=causal, out=out, lse=lse, return_lse=True)
    assert got[0] is out and got[1] is lse and cache.device_status() == 0
    assert torch.all(out[n:] == 9.0) and torch.all(lse[n:] == 9.0)
    ro, rl, info = osv.kv_attention(f64(q[:n]), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, scale, causal)
    keys = max(s.lens + [1])
    e = (D * 2.0 ** -23 + 2.0 ** -21) * info["a"]
    tol = ((2 * e + 2.0 ** -11 + (keys + 66) * 2.0 ** -23)[..., None] * info["pv"]
           + keys * 2.0 ** -25 * info["vmax"][..., None] + HALF[dtype] * np.abs(ro))
    tol = tol + (2.0 ** -25 if dtype is torch.float16 else 0.0)
    err = np.abs(f64(out[:n]) - ro)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    gl = f64(lse[:n])
    dead = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), dead) and np.all(f64(out[:n])[dead] == 0)
    ltol = e + (keys + 64) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(rl, where=~dead, out=np.zeros_like(rl)))
    assert np.all(np.abs(gl - rl, where=~dead, out=np.zeros_like(rl)) <= ltol)
    return out, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_decode(page, D, dtype):
    s = Setup([1] * 7, [0, 1, 15, page - 1, page, 333, 1200], D=D, page=page, seed=10).fill()
    _check_attention(s, dtype, G=4, strided=True)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 24])
def test_attention_group_sizes(G):
    s = Setup([1, 2, 1], [100, 700, 31], H=2, D=64, page=16, seed=11).fill()
    _check_attention(s, torch.bfloat16, G=G)


@pytest.mark.parametrize("D,page,G,causal", [(128, 64, 4, True), (64, 16, 3, True), (128, 32, 1, False), (64, 128, 8, True),
                                             (128, 16, 7, False), (128, 128, 2, True)])
def test_attention_prompts(D, page, G, causal):
    """Chunks of prompts from one token to a few hundred, on contexts from none to long, with
    unused rows behind the last."""
    s = Setup([200, 1, 65, 0, 129, 16], [0, 90, 300, 50, 511, 1], D=D, page=page, seed=12).fill()
    _check_attention(s, torch.bfloat16, G=G, causal=causal, tail=4)


def test_attention_empty_sequences():
    """Sequences of length zero (no rows), and lengths of one; non-causal too."""
    s = Setup([0, 1, 0, 1], [0, 0, 5, 1], D=64, page=16, seed=13).fill()
    for causal in (True, False):
        _check_attention(s, torch.float16, G=2, causal=causal)


def test_attention_split_sequences():
    """One long sequence among short ones: several chunks, joined; and a loose length bound."""
    s = Setup([1, 1, 3], [9000, 40, 2500], H=1, D=64, page=64, seed=14, width=400).fill()
    a = _check_attention(s, torch.bfloat16, G=4)
    b = _check_attention(s, torch.bfloat16, G=4, max_seq_len=400 * 64)
    assert torch.allclose(a[0].float(), b[0].float(), atol=0.02)


def test_attention_scores_of_all_sizes():
    """Flat, peaked, negative and zero scalings; scores in the thousands."""
    s = Setup([1, 40], [500, 300], D=128, page=32, seed=15).fill()
    for scale, gain in ((0.0, 1.0), (1.0, 8.0), (-0.3, 2.0), (1e-6, 1.0), (30.0, 30.0)):
        _check_attention(s, torch.bfloat16, G=2, scale=scale, gain=gain)


def test_attention_units_of_pages_far_apart():
    """Pages whose values of v differ by 2^70, the small ones carrying the probability (a key that
    matches the query in the small page), in both orders."""
    for first in (0, 1):
        s = Setup([1], [95], H=1, D=64, page=16, seed=16).fill()
        small = s.table[0, [1 + first, 4 - first]]
        for p in s.table[0, :6]:
            s.vs[p, 0] = 162
        for p in small:
            s.vs[p, 0] = 92
            s.k[p, 0] = osv.e4m3_encode(np.full((16, 64), 100.0))
            s.ks[p, 0] = 127
        q = torch.full((1, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
        out = s.cache().attention(q, *s.batch(), max_q_len=1, scale=1.0)
        ro, _, info = osv.kv_attention(f64(q), s.k, s.ks, s.v, s.vs, s.cu, s.lens, s.table, 1.0, True)
        assert np.abs(ro).max() < 1e-3  # the large pages have no weight at all
        tol = (2.0 ** -10 + 2.0 ** -14) * info["pv"] + 2.0 ** -8 * np.abs(ro)
        assert np.all(np.abs(f64(out) - ro) <= tol)


def test_attention_queries_of_far_apart_sizes():
    """Rows of q scaled from 2^-60 to 2^60 (scores scaled back), and zero queries."""
    s = Setup([6], [70], H=1, D=128, page=32, seed=17).fill()
    base = torch.randn(6, 1, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    base[5] = 0
    cache = s.cache()
    want = cache.attention(base.cuda(), *s.batch(), max_q_len=6, scale=0.1)
    for e in (-60, -20, 20, 60):
        got = cache.attention((base * 2.0 ** e).cuda(), *s.batch(), max_q_len=6, scale=0.1 * 2.0 ** -e)
        assert torch.equal(got, want)


def test_attention_stale_and_missing_pages():
    """Codes behind the last token are NaN patterns throughout these tests (Setup); a page outside
    the cache is skipped and reported, the rest computed."""
    s = Setup([1, 1], [100, 60], H=2, D=64, page=16, seed=18).fill()
    cache = s.cache()
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    cu, lens, table = s.batch()
    for bad in (-1, s.pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out, lse = cache.attention(q, cu, lens, t, max_q_len=1, scale=0.125, return_lse=True)
        assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
        keep = [j for j in range(101) if j // 16 != 2]
        k, v = osv.kv_values(s.k, s.ks, s.table[0], 101)[keep], osv.kv_values(s.v, s.vs, s.table[0], 101)[keep]
        z = 0.125 * np.einsum("jhd,hgd->hgj", k, f64(q[0]).reshape(2, 2, 64))
        assert np.allclose(f64(lse[0]).reshape(2, 2), np.log(np.exp(z).sum(-1)), atol=1e-5)
        p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
        assert np.allclose(f64(out[0]).reshape(2, 2, 64), np.einsum("hgj,jhd->hgd", p, v), rtol=2.0 ** -7, atol=2e-3)


def test_attention_bad_batches_are_refused():
    s = Setup([1, 2], [50, 20], H=1, D=64, page=16, seed=19).fill()
    q = torch.randn(3, 2, 64, device="cuda").half()

    def run(change, **kw):
        cu, lens, table = (x.cpu().clone() for x in s.batch())
        change(cu, lens)
        cache = s.cache()
        out = torch.full((3, 2, 64), 5.0, dtype=torch.float16, device="cuda")
        a = dict(max_q_len=2)
        a.update(kw)
        cache.attention(q, cu.cuda(), lens.cuda(), table.cuda(), out=out, **a)
        assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
        return (out != 5.0).flatten(1).any(1).tolist()

    assert run(lambda cu, lens: lens.__setitem__(0, 1000)) == [False, True, True]
    assert run(lambda cu, lens: lens.__setitem__(1, 1)) == [True, False, False]
    assert run(lambda cu, lens: lens.__setitem__(1, -5)) == [True, False, False]
    assert run(lambda cu, lens: cu.__setitem__(2, 9)) == [True, False, False]
    assert run(lambda cu, lens: None, max_seq_len=30) == [False, True, True]


def test_attention_streams_and_graphs():
    """Another stream; two captured graphs replayed at once with new contents of the batch."""
    s = Setup([1, 1, 1], [5000, 900, 3], H=2, D=128, page=64, seed=20).fill()
    cache = s.cache()
    cu, lens, table = s.batch()
    q = torch.randn(3, 8, 128, device="cuda").to(torch.bfloat16)
    call = lambda **kw: cache.attention(q, cu, lens, table, max_q_len=1, **kw)  # noqa: E731
    want = call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    call(out=out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    lens.copy_(_i32([4000, 901, 2]))
    want = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, x in zip(graphs, streams):
            with torch.cuda.stream(x):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_cache_past_four_gigabytes():
    """Pages whose codes lie past 2^32 bytes are written and read."""
    H, D, page = 8, 128, 128
    pages = (1 << 32) // (H * D * page) + 40
    cache = KVCache(pages, page, H, D)
    table = _i32([[pages - 1, 7, pages - 3]])
    n = 2 * page + 9
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    cache.append(k, v, _i32([0, n]), _i32([n]), table)
    q = torch.randn(1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    out = cache.attention(q, _i32([0, 1]), _i32([n]), table, max_q_len=1)
    assert cache.device_status() == 0
    kk, vv = f64(k), f64(v)
    z = np.einsum("jhd,hd->hj", kk, f64(q)[0]) * D ** -0.5
    p = np.exp(z - z.max(1, keepdims=True))
    want = np.einsum("hj,jhd->hd", p / p.sum(1, keepdims=True), vv)
    assert np.abs(f64(out)[0] - want).max() < 0.05  # E4M3 keys and values: 2^-4 each, averaged


def test_python_refusals():
    s = Setup([1], [3], H=2, D=64, page=16).fill()
    cache, (cu, lens, table) = s.cache(), s.batch()
    k = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    bad = [lambda: cache.append(k.float(), k, cu, lens, table), lambda: cache.append(k, k.bfloat16(), cu, lens, table),
           lambda: cache.append(k[:, :1], k, cu, lens, table), lambda: cache.append(k, k, cu.long(), lens, table),
           lambda: cache.append(k, k, cu[:1], lens, table), lambda: cache.append(k, k, cu, lens, table[0]),
           lambda: cache.append(k, k, cu, lens, table, q_out=q), lambda: cache.append(k.transpose(1, 2), k, cu, lens, table),
           lambda: cache.append(k, k, cu, lens, table, q=q, q_out=q[:, :2].contiguous()),
           lambda: cache.attention(q.float(), cu, lens, table, 1), lambda: cache.attention(q[..., :32], cu, lens, table, 1),
           lambda: cache.attention(q, cu.cpu(), lens, table, 1),
           lambda: cache.attention(q, cu, lens, table, 1, lse=torch.zeros(1, 4, device="cuda").half()),
           lambda: KVCache(4, 24, 2, 64), lambda: KVCache(4, 16, 2, 80)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in [lambda: cache.attention(q[:, :3].contiguous(), cu, lens, table, 1),
              lambda: cache.attention(q, cu, lens, table, 2), lambda: cache.attention(q, cu, lens, table, 1, max_seq_len=17),
              lambda: cache.append(k, k, cu, lens, table, inv_freq=torch.ones(9, device="cuda"))]:
        with pytest.raises(FQError):
            f()


# ------------------------------------------------------------------------------------
# the path together
# ------------------------------------------------------------------------------------
def test_prompt_and_decode_steps_together():
    """A rotated INT8 projection to q, k, v, rotary appending and attention: a prompt in two
    chunks and then single tokens must give what one pass over the whole sequence gives, within
    what the pages' growing exponents may change; every output is checked against the oracle on
    the cache's own contents."""
    H, G, D, page, M, N = 2, 2, 64, 16, 16, 32
    Hq, O, n = H * G, (H * G + 2 * H) * D, 45
    g = np.random.default_rng(21)
    x = torch.from_numpy(g.standard_normal((n, M, N), dtype=np.float32)).to(torch.bfloat16).cuda()
    P = [torch.from_numpy(np.linalg.qr(g.standard_normal((k, k)))[0].copy()).to(torch.bfloat16).cuda() for k in (M, N)]
    w = torch.from_numpy(g.integers(-127, 128, (O, M * N), dtype=np.int8)).cuda()
    sw = torch.full((O,), 6e-4, device="cuda")
    f = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    table = _i32([[2, 0, 3]])

    def steps(sizes):
        cache, outs, at = KVCache(4, page, H, D), [], 0
        for c in sizes:
            codes, qs = FlatQuant(c, M, N).quantize_per_token(x[at:at + c].contiguous(), *P, out_dtype="int8")
            qkv = int8_matmul(codes, qs, w, sw).view(c, Hq + 2 * H, D)
            at += c
            batch = (_i32([0, c]), _i32([at]), table)
            q = cache.append(qkv[:, Hq:Hq + H], qkv[:, Hq + H:], *batch, q=qkv[:, :Hq], inv_freq=f)
            out = cache.attention(q, *batch, max_q_len=c)
            assert cache.device_status() == 0
            ro, _, info = osv.kv_attention(f64(q), _codes(cache.k), cache.k_scale.cpu().numpy(), _codes(cache.v),
                                           cache.v_scale.cpu().numpy(), [0, c], [at], table.tolist(), D ** -0.5, True)
            e = (D * 2.0 ** -23 + 2.0 ** -21) * info["a"]
            tol = (2 * e + 2.0 ** -11 + 2.0 ** -16)[..., None] * info["pv"] + 2.0 ** -19 * info["vmax"][..., None]
            assert np.all(np.abs(f64(out) - ro) <= tol + 2.0 ** -8 * np.abs(ro))
            outs.append(out)
        return torch.cat(outs).float()

    whole, parts = steps([n]), steps([30, 9, 1, 1, 1, 1, 1, 1])
    rms = whole.square().mean().sqrt()
    assert (whole - parts).square().mean().sqrt() < 2.0 ** -4 * rms  # one E4M3 step of keys and values


# ------------------------------------------------------------------------------------
# the tensor-core attention kernel (sequences with more than 64 rows)
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("n", [17, 64, 65, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_row_tile_edges(n, D):
    """Row counts around one and two row tiles of 128, alone and beside a decode step."""
    for new, ctx in (([n], [0]), ([n, 1], [100, 40])):
        s = Setup(new, ctx, H=1, D=D, page=64, seed=30).fill()
        _check_attention(s, torch.bfloat16, G=1)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_key_step_edges(page, D, causal):
    """Lengths around the 128-key steps, with pages that end inside one."""
    s = Setup([70, 128, 90, 130], [1, 0, 167, 255], H=2, D=D, page=page, seed=31).fill()
    _check_attention(s, torch.float16, G=2, causal=causal, strided=True)


def test_attention_split_prompts():
    """A short prompt on a long context is divided into chunks of keys and joined."""
    s = Setup([40, 3], [5000, 2100], H=1, D=128, page=64, seed=32).fill()
    _check_attention(s, torch.bfloat16, G=2)
    s = Setup([90], [3000], H=1, D=64, page=16, seed=33).fill()
    _check_attention(s, torch.float16, G=1)


def test_attention_prompt_page_exponents():
    """Pages whose exponents differ by up to 2^30 within one 128-key step."""
    s = Setup([80], [300], H=1, D=128, page=16, seed=34).fill()
    rng = np.random.default_rng(5)
    for p in s.table[0]:
        s.vs[p, 0] = 127 + rng.integers(-15, 16)
        s.ks[p, 0] = min(s.ks[p, 0], 120) - rng.integers(0, 25)
    _check_attention(s, torch.bfloat16, G=1)


def test_attention_prompt_missing_page():
    s = Setup([70], [200], H=1, D=64, page=16, seed=35).fill()
    cache = s.cache()
    q = torch.randn(70, 2, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    cu, lens, table = s.batch()
    t = table.clone()
    t[0, 3] = s.pages + 5
    out, lse = cache.attention(q, cu, lens, t, max_q_len=70, scale=0.125, return_lse=True)
    assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
    k, v = osv.kv_values(s.k, s.ks, s.table[0], 270)[:, 0], osv.kv_values(s.v, s.vs, s.table[0], 270)[:, 0]
    for i in (0, 33, 69):
        keep = [j for j in range(200 + i + 1) if j // 16 != 3]
        z = 0.125 * f64(q[i]) @ k[keep].T
        assert np.allclose(f64(lse[i]), np.log(np.exp(z).sum(-1)), atol=1e-5)
        p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
        assert np.allclose(f64(out[i]), p @ v[keep], rtol=2.0 ** -7, atol=2e-3)


def test_attention_loose_bounds():
    """max_q_len and max_seq_len above what the batch has give the same result."""
    s = Setup([70, 2, 1], [100, 300, 0], H=2, D=128, page=32, seed=36, width=100).fill()
    cache = s.cache()
    q = torch.randn(73, 4, 128, device="cuda").to(torch.bfloat16)
    a = cache.attention(q, *s.batch(), max_q_len=70, max_seq_len=302)
    b = cache.attention(q, *s.batch(), max_q_len=73, max_seq_len=3200)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * a.float().abs().max()
    one = Setup([3], [50], H=1, D=64, page=16, seed=37).fill()
    q = torch.randn(200, 2, 64, device="cuda").half()
    a = one.cache().attention(q, *one.batch(), max_q_len=3)
    b = one.cache().attention(q, *one.batch(), max_q_len=200)
    assert (a[:3].float() - b[:3].float()).abs().max() <= 2.0 ** -9 * a[:3].float().abs().max()


def test_memory_of_the_given_stream():
    """Outputs and workspaces of a call on another stream are not memory that the current stream
    has freed but still has to read."""
    s = Setup([1], [5000], H=1, D=64, page=64, seed=60).fill()
    cache, (cu, lens, table) = s.cache(), s.batch()
    q = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16)
    a = torch.ones(3, 64, dtype=torch.int8, device="cuda")
    sc = torch.ones(3, device="cuda")
    fq, x = FlatQuant(3, 16, 16), torch.randn(3, 16, 16, device="cuda").to(torch.bfloat16)
    eye = torch.eye(16, device="cuda").to(torch.bfloat16)
    st = torch.cuda.Stream()
    calls = [lambda: cache.attention(q, cu, lens, table, 1, return_lse=True, stream=st),
             lambda: cache.append(k, k, cu, lens, table, q=q, stream=st),
             lambda: int8_matmul(a, sc, a, sc, stream=st),
             lambda: fq.quantize_per_token(x, eye, eye, out_dtype="int8", stream=st)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (8, 256, 1024, 4096, 16384, 65536)
                for _ in range(64)]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # about 20 ms
        copies = [h.clone() for h in held]
        del held  # free, and read by the copies that are still queued
        call()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies)


@pytest.mark.parametrize("G,D,causal", [(1, 128, True), (4, 64, True), (8, 128, False), (16, 64, True)])
def test_attention_few_chunks(G, D, causal):
    """Two to eight chunks of a sequence, beside sequences of one chunk and of none."""
    s = Setup([1, 1, 0, 2, 1, 1], [299, 1023, 0, 1500, 256, 0], H=2, D=D, page=64, seed=61).fill()
    _check_attention(s, torch.bfloat16, G, causal=causal, tail=2)
    _check_attention(s, torch.float16, G, causal=causal, max_seq_len=s.width * 64)


def test_attention_few_chunks_of_many_sequences():
    """More sequences and heads than one wave of CTAs, the longest of a few chunks."""
    ctx = [3, 0, 70] * 19 + [4200, 2047, 2048]
    s = Setup([1] * 60, ctx, H=8, D=128, page=128, seed=62).fill()
    _check_attention(s, torch.bfloat16, 1)


def test_attention_chunk_with_a_page_outside():
    """A page outside the cache in one of a sequence's chunks: its keys are left out, the others join."""
    s = Setup([1], [899], H=1, D=64, page=16, seed=63).fill()
    cache = s.cache()
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    cu, lens, table = s.batch()
    t = table.clone()
    t[0, 20:36] = -7  # the second chunk's pages, all of them
    out, lse = cache.attention(q, cu, lens, t, max_q_len=1, scale=0.125, return_lse=True)
    assert cache.device_status() == _lib.FQ_KV_BAD_BATCH
    k, v = osv.kv_values(s.k, s.ks, s.table[0], 900)[:, 0], osv.kv_values(s.v, s.vs, s.table[0], 900)[:, 0]
    keep = [j for j in range(900) if not 20 <= j // 16 < 36]
    z = 0.125 * f64(q[0]) @ k[keep].T
    assert np.allclose(f64(lse[0]), np.log(np.exp(z).sum(-1)), atol=1e-5)
    p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
    assert np.allclose(f64(out[0]), p @ v[keep], rtol=2.0 ** -7, atol=2e-3)


@pytest.mark.parametrize("new,ctx,longest", [([1, 1, 2], [1500, 700, 90], 1600), ([40, 1, 30], [900, 2500, 0], 2600)])
def test_graphs_replayed_with_other_lengths(new, ctx, longest):
    """Two graphs of one cache (chunks joined in clusters; a prompt and decode steps in one call)
    replayed at the same time with other lengths and pages, and a third call beside them."""
    s = Setup(new, ctx, H=2, D=128, page=32, seed=64, width=-(-longest // 32)).fill()
    cache = s.cache()
    cu, lens, table = s.batch()
    q = torch.randn(sum(new), 8, 128, device="cuda").to(torch.bfloat16)
    call = lambda: cache.attention(q, cu, lens, table, max(new), max_seq_len=longest, return_lse=True)  # noqa: E731
    call()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call())
        graphs.append(gr)
    lens.copy_(_i32([n + c // 3 for n, c in zip(new, ctx)]))
    table.copy_(table[:, torch.arange(table.shape[1] - 1, -1, -1)].clone().clamp_(min=0))
    want = call()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, x in zip(graphs, streams):
            with torch.cuda.stream(x):
                gr.replay()
        again = call()
    torch.cuda.synchronize()
    assert cache.device_status() == 0
    bits = lambda x: x.view(torch.uint8)  # noqa: E731  (the turned tables reach NaN codes)
    for o, l in outs + [again]:
        assert torch.equal(bits(o), bits(want[0])) and torch.equal(bits(l), bits(want[1]))


def test_append_in_place_of_the_queries():
    """q_out may be q itself."""
    s = Setup([3, 40], [5, 0], H=2, D=64, page=16, seed=65)
    cu, lens, table = s.batch()
    k = torch.randn(43, 2, 64, device="cuda").half()
    q = torch.randn(43, 12, 64, device="cuda").half()
    f = torch.rand(32, device="cuda")
    want = s.cache().append(k, k, cu, lens, table, q=q, inv_freq=f)
    got = s.cache().append(k, k, cu, lens, table, q=q, inv_freq=f, q_out=q)
    assert got is q and torch.equal(got, want)
