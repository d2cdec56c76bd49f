"""The 8-bit serving operators as cases to measure: the rotated INT8 linear layer (per-token
rotate + quantize, then the INT8 product), the INT8 product alone, appending rotary-encoded
keys and values to the 8-bit paged cache, and attention over that cache.

Each case is a dict of plain values. `prepare` makes inputs on the GPU from a seed, `run`
makes one pass (plain torch operations, or the library's calls where `own` is true), `work`
counts what a pass cannot do without, `exact` gives the result in 64 bits.
"""

import math
import random

import torch

own = False

PAGE_EXP_MIN, PAGE_EXP_MAX = -40, 40  # range of a page's shared exponent
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def listed():
    return [
        # a rotated linear layer of a decode step: 16 sequences, hidden size 64 x 64
        {"name": "linear_decode", "op": "linear", "tokens": 16, "M": 64, "N": 64, "O": 6144,
         "dtype": "bf16", "clip": 1.0},
        # the same layer in prefill, at the row length of the largest rotate workload (128 x 112)
        {"name": "linear_prefill", "op": "linear", "tokens": 4096, "M": 128, "N": 112, "O": 4096,
         "dtype": "bf16", "clip": 0.95},
        # one token through a wide projection: the weights are read once for one row
        {"name": "matmul_one_token", "op": "matmul", "tokens": 1, "O": 14336, "L": 4096, "out": "bf16"},
        # a ragged batch with an output width that is no multiple of a tile or a vector
        {"name": "matmul_ragged", "op": "matmul", "tokens": 333, "O": 4099, "L": 8192, "out": "fp16"},
        # prefill at the sizes of the FP4 product that bench.py times
        {"name": "matmul_prefill", "op": "matmul", "tokens": 8192, "O": 4096, "L": 14336, "out": "bf16"},
        # one new token of each of 64 running sequences
        {"name": "append_decode", "op": "append", "seqs": 64, "new_min": 1, "new_max": 1,
         "ctx_min": 1, "ctx_max": 4000, "kv_heads": 8, "group": 4, "D": 128, "page": 64,
         "rot": 128, "interleaved": False, "base": 500000.0, "dtype": "bf16", "lens": 1},
        # ragged prompts on top of cached prefixes that end inside a page, half of the head rotated
        {"name": "append_prefill", "op": "append", "seqs": 7, "new_min": 300, "new_max": 2500,
         "ctx_min": 0, "ctx_max": 500, "kv_heads": 8, "group": 4, "D": 128, "page": 16,
         "rot": 64, "interleaved": True, "base": 10000.0, "dtype": "fp16", "lens": 2},
        # one short conversation: latency
        {"name": "attention_one_short", "op": "attention", "seqs": 1, "q_min": 1, "q_max": 1,
         "ctx_min": 700, "ctx_max": 700, "kv_heads": 8, "group": 4, "D": 128, "page": 64,
         "causal": True, "dtype": "bf16", "lens": 3},
        # a full decode batch of unequal contexts
        {"name": "attention_decode_batch", "op": "attention", "seqs": 64, "q_min": 1, "q_max": 1,
         "ctx_min": 500, "ctx_max": 16000, "kv_heads": 8, "group": 8, "D": 128, "page": 64,
         "causal": True, "dtype": "bf16", "lens": 4},
        # two very long documents, small pages, small heads, few heads
        {"name": "attention_long", "op": "attention", "seqs": 2, "q_min": 1, "q_max": 1,
         "ctx_min": 150000, "ctx_max": 260000, "kv_heads": 4, "group": 7, "D": 64, "page": 16,
         "causal": True, "dtype": "fp16", "lens": 5},
        # prompt chunks on top of cached prefixes
        {"name": "attention_chunks", "op": "attention", "seqs": 5, "q_min": 200, "q_max": 1100,
         "ctx_min": 1000, "ctx_max": 6000, "kv_heads": 8, "group": 4, "D": 128, "page": 32,
         "causal": True, "dtype": "bf16", "lens": 6},
        # one whole long prompt
        {"name": "attention_prefill", "op": "attention", "seqs": 1, "q_min": 8192, "q_max": 8192,
         "ctx_min": 0, "ctx_max": 0, "kv_heads": 8, "group": 4, "D": 128, "page": 64,
         "causal": True, "dtype": "bf16", "lens": 7},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "matmul", "append", "attention", "attention"])
    if op == "linear":
        M, N = rng.choice([(16, 16), (64, 64), (64, 80), (32, 112), (64, 128), (128, 112), (128, 128)])
        return {"op": op, "tokens": _log(rng, 1, 4096), "M": M, "N": N, "O": _log(rng, 64, 8192),
                "dtype": rng.choice(["bf16", "fp16"]), "clip": rng.choice([0.9, 0.95, 1.0])}
    if op == "matmul":
        return {"op": op, "tokens": _log(rng, 1, 8192), "O": _log(rng, 64, 8192),
                "L": 16 * _log(rng, 16, 512), "out": rng.choice(["bf16", "fp16", "fp32"])}
    heads = {"kv_heads": rng.choice([1, 2, 4, 8]), "group": rng.choice([1, 2, 3, 4, 7, 8]),
             "D": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]),
             "dtype": rng.choice(["bf16", "fp16"]), "lens": rng.randrange(1 << 20)}
    if op == "append":
        if rng.random() < 0.5:  # decode steps
            size = {"seqs": _log(rng, 1, 256), "new_min": 1, "new_max": rng.choice([1, 1, 4])}
        else:
            size = {"seqs": _log(rng, 1, 8), "new_min": 1, "new_max": _log(rng, 16, 1500)}
        return {"op": op, **size, "ctx_min": 0, "ctx_max": _log(rng, 16, 4000), **heads,
                "rot": rng.choice([heads["D"], heads["D"] // 2]), "interleaved": rng.random() < 0.5,
                "base": rng.choice([10000.0, 500000.0])}
    if rng.random() < 0.6:  # decode steps, a few tokens at most
        seqs = _log(rng, 1, 64)
        size = {"seqs": seqs, "q_min": 1, "q_max": rng.choice([1, 1, 3]), "ctx_min": 0,
                "ctx_max": _log(rng, 64, 200000 // seqs + 200)}
    else:
        size = {"seqs": _log(rng, 1, 4), "q_min": 1, "q_max": _log(rng, 32, 1500), "ctx_min": 0,
                "ctx_max": _log(rng, 16, 4000)}
    return {"op": op, **size, **heads, "causal": rng.random() < 0.8}


def _lengths(case):
    """(new tokens, total length) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    key = "new" if case["op"] == "append" else "q"
    got = []
    for _ in range(case["seqs"]):
        n = r.randint(case[key + "_min"], case[key + "_max"])
        got.append((n, n + r.randint(case["ctx_min"], case["ctx_max"])))
    return got


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _page_exponent(amax):
    """Smallest e with amax <= 448 * 2^e, clamped (in 64 bits, so that no quotient rounds)."""
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax > 0, e, PAGE_EXP_MIN).clamp(PAGE_EXP_MIN, PAGE_EXP_MAX).to(torch.int32)


def _filled_cache(gen, pages, H, page, D):
    """A cache in use: values with a few strong channels, a different gain for each page."""
    dev = gen.device
    gain = torch.exp(0.5 * torch.randn(D, generator=gen, device=dev))
    x = torch.randn(pages, H, page, D, generator=gen, device=dev, dtype=torch.bfloat16)
    x *= gain.to(torch.bfloat16)
    x *= torch.exp(0.5 * torch.randn(pages, H, 1, 1, generator=gen, device=dev)).to(torch.bfloat16)
    e = _page_exponent(x.abs().amax(dim=(2, 3)).float())
    x *= torch.exp2(-e.float())[..., None, None].to(torch.bfloat16)
    return x.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _orthogonal(gen, n, dtype):
    g = torch.randn(n, n, generator=gen, device=gen.device, dtype=torch.float64)
    q, r = torch.linalg.qr(g)
    return (q * torch.sign(torch.diagonal(r))).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("linear", "matmul"):
        O = case["O"]
        L = case["M"] * case["N"] if op == "linear" else case["L"]
        s["w"] = torch.randint(-127, 128, (O, L), generator=gen, device=dev, dtype=torch.int8)
        s["w_scale"] = 0.5e-3 + 1e-3 * torch.rand(O, generator=gen, device=dev)
        if op == "linear":
            dt = DTYPES[case["dtype"]]
            x = torch.randn(case["tokens"], case["M"], case["N"], generator=gen, device=dev)
            hot = torch.randint(0, L, (8,), generator=gen, device=dev)
            x.view(case["tokens"], L)[:, hot] *= 20.0  # outlier channels
            s["x"] = x.to(dt)
            s["P1"], s["P2"] = _orthogonal(gen, case["M"], dt), _orthogonal(gen, case["N"], dt)
        else:
            s["a"] = torch.randint(-127, 128, (case["tokens"], L), generator=gen, device=dev, dtype=torch.int8)
            s["a_scale"] = 1e-2 + 3e-2 * torch.rand(case["tokens"], generator=gen, device=dev)
        return s
    lens = _lengths(case)
    B, page, H, D = len(lens), case["page"], case["kv_heads"], case["D"]
    need = [-(-total // page) for _, total in lens]
    pages = 1 + sum(need)  # page 0 belongs to nobody
    order = 1 + torch.randperm(pages - 1, generator=gen, device=dev, dtype=torch.int32)
    width = max(need)
    at = torch.tensor([[sum(need[:b]) + j if j < need[b] else -1 for j in range(width)] for b in range(B)],
                      dtype=torch.int64, device=dev) if B * width < 200000 else None
    if at is None:
        j = torch.arange(width, device=dev)[None, :]
        n = torch.tensor(need, device=dev)[:, None]
        at = torch.where(j < n, torch.cumsum(n, 0) - n + j, -1)
    s["table"] = torch.where(at >= 0, order[at.clamp_min(0)], 0).to(torch.int32).contiguous()
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor([t for _, t in lens], dtype=torch.int32, device=dev)
    s["max_new"], s["max_len"] = max(n for n, _ in lens), max(t for _, t in lens)
    s["k_cache"], s["k_scale"] = _filled_cache(gen, pages, H, page, D)
    s["v_cache"], s["v_scale"] = _filled_cache(gen, pages, H, page, D)
    dt = DTYPES[case["dtype"]]
    Hq = H * case["group"]
    if op == "append":
        # q, k and v as they leave one fused projection: rows of [Hq + 2 H] heads
        qkv = torch.randn(T, Hq + 2 * H, D, generator=gen, device=dev)
        qkv *= torch.exp(0.7 * torch.randn(T, Hq + 2 * H, 1, generator=gen, device=dev))
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["inv_freq"] = (case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev)
                                          / case["rot"])).float()
    else:
        s["q"] = (2.0 * torch.randn(T, Hq, D, generator=gen, device=dev)).to(dt)
        s["scale"] = D ** -0.5
    return s


# ------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------
def _run_own(s):
    import rotation_bit_quantization_token_b200 as fq
    case = s["case"]
    op = case["op"]
    if op == "matmul":
        return fq.int8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], out_dtype=DTYPES[case["out"]])
    if op == "linear":
        if "plan" not in s:
            s["plan"] = (fq.FlatQuant(case["tokens"], case["M"], case["N"], s["x"].dtype),
                         s["P1"].contiguous(), s["P2"].contiguous())
        plan, P1, P2 = s["plan"]
        codes, qs = plan.quantize_per_token(s["x"], P1, P2, clip_ratio=case["clip"], out_dtype="int8")
        return fq.int8_matmul(codes, qs, s["w"], s["w_scale"], out_dtype=s["x"].dtype), qs
    if "plan" not in s:
        s["plan"] = fq.KVCache.from_buffers(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    cache = s["plan"]
    if op == "append":
        q = cache.append(s["k"], s["v"], s["cu"], s["seq_lens"], s["table"], q=s["q"], inv_freq=s["inv_freq"],
                         interleaved=case["interleaved"])
        return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return cache.attention(s["q"], s["cu"], s["seq_lens"], s["table"], max_q_len=s["max_new"],
                           max_seq_len=s["max_len"], scale=s["scale"], causal=case["causal"], return_lse=True)


# ------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------
def _plain_matmul(a, a_scale, w, w_scale, dtype):
    # sums of 8-bit products pass 2^24: in 64 bits they are exact
    acc = torch.matmul(a.double(), w.double().t()).float()
    return (acc * a_scale[:, None] * w_scale[None, :]).to(dtype)


def _plain_linear(s):
    case, x = s["case"], s["x"].float()
    r = torch.matmul(s["P1"].float(), torch.matmul(x, s["P2"].float())).reshape(x.shape[0], -1)
    qs = r.abs().amax(dim=1) / (127.0 / case["clip"])
    inv = torch.where(qs > 0, 1.0 / qs, torch.zeros_like(qs))
    codes = torch.round(r * inv[:, None]).clamp(-128, 127)
    return _plain_matmul(codes, qs, s["w"], s["w_scale"], s["x"].dtype), qs


def _token_of(s, T):
    """Sequence and index within the sequence's new tokens, for each row."""
    t = torch.arange(T, device=s["cu"].device)
    b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    return b, t - s["cu"].long()[b]


def _plain_rotate(x, pos, inv_freq, interleaved):
    rot = 2 * inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((r, y[..., rot:]), dim=-1)


def _plain_store(cache, scale, x, pages, rows, older, t):
    """New rows x [T, H, D] (`rows`, from index t) into the pages [B, P] they fall in; a page's older
    rows move to its new exponent, every other row stays as it is."""
    codes = cache.view(torch.uint8)
    new = x[t.clamp(0, x.shape[0] - 1)] * rows[..., None, None]                # [B, P, page, H, D]
    e = _page_exponent(new.abs().amax(dim=(2, 4)))                              # [B, P, H]
    old_e = scale[pages].int() - 127
    e = torch.where(older.any(dim=2)[..., None], torch.maximum(e, old_e), e)
    e = torch.where(rows.any(dim=2)[..., None], e, old_e)
    old = codes[pages]                                                          # [B, P, H, page, D]
    moved = old.view(cache.dtype).float() * torch.exp2((old_e - e).float())[..., None, None]
    put = new.permute(0, 1, 3, 2, 4) * torch.exp2(-e.float())[..., None, None]
    both = torch.where(rows[:, :, None, :, None], put, moved).clamp(-E4M3_MAX, E4M3_MAX)
    both = both.to(cache.dtype).view(torch.uint8)
    codes[pages] = torch.where((rows | older)[:, :, None, :, None], both, old)
    scale[pages] = (e + 127).to(torch.uint8)


def _plain_append(s):
    case, T = s["case"], s["k"].shape[0]
    page = case["page"]
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    n = cu[1:] - cu[:-1]
    first = lens - n
    b, i = _token_of(s, T)
    pos = first[b] + i
    P = (s["max_new"] + page - 2) // page + 1  # pages that so many tokens can touch
    j = first[:, None] // page + torch.arange(P, device=cu.device)[None, :]
    there = (j * page < lens[:, None]) & (n[:, None] > 0)
    pages = torch.where(there, s["table"].long().gather(1, j.clamp(max=s["table"].shape[1] - 1)), 0)
    at = (j * page)[:, :, None] + torch.arange(page, device=cu.device)          # positions of the pages' rows
    rows = (at >= first[:, None, None]) & (at < lens[:, None, None]) & there[:, :, None]
    t = cu[:-1, None, None] + at - first[:, None, None]
    older = (at < first[:, None, None]) & there[:, :, None]
    k = _plain_rotate(s["k"], pos, s["inv_freq"], case["interleaved"])
    _plain_store(s["k_cache"], s["k_scale"], k, pages, rows, older, t)
    _plain_store(s["v_cache"], s["v_scale"], s["v"].float(), pages, rows, older, t)
    q = _plain_rotate(s["q"], pos, s["inv_freq"], case["interleaved"]).to(s["q"].dtype)
    return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_values(cache, scale, table):
    """The cached values of every sequence, [B, H, positions, D]."""
    x = cache[table].float() * torch.exp2(scale[table].float() - 127.0)[..., None, None]
    B, P, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * page, D)


def _plain_attention(s):
    case, q = s["case"], s["q"]
    H, G, D = case["kv_heads"], case["group"], case["D"]
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    B, Q, T = lens.numel(), s["max_new"], q.shape[0]
    i = torch.arange(Q, device=q.device)
    rows = q[(cu[:-1, None] + i).clamp(max=T - 1)].float()                      # [B, Q, H G, D]
    rows = rows.reshape(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    table = s["table"].long()
    p = torch.matmul(rows, _plain_values(s["k_cache"], s["k_scale"], table).transpose(2, 3))
    p *= s["scale"]
    last = lens[:, None] if not case["causal"] else lens[:, None] - (cu[1:] - cu[:-1])[:, None] + i + 1
    key = torch.arange(p.shape[-1], device=q.device)
    hidden = key >= torch.minimum(last, lens[:, None])[..., None]               # [B, 1 or Q, keys]
    p = p.view(B, H, Q, G, -1).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = p.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]                                      # -inf where nothing is seen
    p /= torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p.view(B, H, Q * G, -1), _plain_values(s["v_cache"], s["v_scale"], table)).view(B, H, Q, G, D)
    b, i = _token_of(s, T)
    out = o.permute(0, 2, 1, 3, 4)[b, i].reshape(T, H * G, D).to(q.dtype)
    return out, lse.permute(0, 2, 1, 3)[b, i].reshape(T, H * G)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "matmul":
        return _plain_matmul(state["a"], state["a_scale"], state["w"], state["w_scale"], DTYPES[case["out"]])
    if op == "linear":
        return _plain_linear(state)
    return _plain_append(state) if op == "append" else _plain_attention(state)


# ------------------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("linear", "matmul"):
        T, O = case["tokens"], case["O"]
        L = case["M"] * case["N"] if op == "linear" else case["L"]
        out = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype" if op == "linear" else "out"]]
        by = O * L + 4 * O + T * O * out + 4 * T
        fl = 2.0 * T * O * L
        if op == "linear":
            by += 2 * T * L + 2 * (case["M"] ** 2 + case["N"] ** 2)
            fl += 2.0 * T * L * (case["M"] + case["N"])
        else:
            by += T * L
        return {"bytes": by, "flops": fl}
    lens = _lengths(case)
    H, G, D, page = case["kv_heads"], case["group"], case["D"], case["page"]
    T = sum(n for n, _ in lens)
    meta = 4 * (2 * len(lens) + 1)
    if op == "append":
        touched = sum((t - 1) // page - (t - n) // page + 1 for n, t in lens if n)
        by = T * H * D * 6 + T * H * G * D * 4 + touched * (2 * H + 4) + meta + 2 * case["rot"]
        return {"bytes": by, "flops": T * H * (G + 1) * case["rot"] * 3.0 + T * H * D * 4.0}
    pages = sum(-(-t // page) for _, t in lens)
    by = sum(t for _, t in lens) * H * D * 2 + pages * (2 * H + 4) + T * H * G * (4 * D + 4) + meta
    seen = sum(sum(t - n + 1 + i for i in range(n)) if case["causal"] else n * t for n, t in lens)
    return {"bytes": by, "flops": 4.0 * D * H * G * seen}


def _exact_rotate(x, pos, f, interleaved):
    x = x.double().clone()
    ang = pos[:, None].double() * f.double()[None, :]
    half = f.numel()
    lo = torch.arange(half, device=x.device) * 2 if interleaved else torch.arange(half, device=x.device)
    hi = lo + 1 if interleaved else lo + half
    z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.ones_like(ang), ang)[:, None, :]
    x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _e4m3(x):
    """Nearest e4m3 value (ties to the even code) of |x| <= 448, in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "matmul"):
        dt = DTYPES[case["dtype" if op == "linear" else "out"]]
        if op == "matmul":
            a, sa = s["a"].double(), s["a_scale"].double()
        else:
            r = torch.einsum("im,kmn->kin", s["P1"].double(), torch.einsum("kmj,jn->kmn", s["x"].double(), s["P2"].double()))
            r = r.reshape(r.shape[0], -1)
            sa = r.abs().amax(1) * case["clip"] / 127.0
            a = torch.round(r / torch.where(sa > 0, sa, 1.0)[:, None]).clamp(-128, 127)
        C = torch.einsum("tl,ol->to", a, s["w"].double()) * sa[:, None] * s["w_scale"].double()
        return C if op == "matmul" else (C, sa)
    lens = _lengths(case)
    page, H, G, D = case["page"], case["kv_heads"], case["group"], case["D"]
    cu = s["cu"].tolist()
    if op == "append":
        table = s["table"].tolist()
        pos = torch.cat([torch.arange(t - n, t) for n, t in lens]).to(s["q"].device)
        q = _exact_rotate(s["q"], pos, s["inv_freq"], case["interleaved"])
        k = _exact_rotate(s["k"], pos, s["inv_freq"], case["interleaved"])
        back = []
        for cache, sc, x in ((s["k_cache"], s["k_scale"], k), (s["v_cache"], s["v_scale"], s["v"].double())):
            vals, exps = cache.double(), sc.int() - 127
            for b, (n, t) in enumerate(lens):
                at = t - n
                while at < t:
                    end = min(t, (at // page + 1) * page)
                    pg = table[b][at // page]
                    rows = x[cu[b] + at - (t - n):cu[b] + end - (t - n)].permute(1, 0, 2)  # [H, rows, D]
                    amax = rows.abs().amax(dim=(1, 2))
                    e = torch.ceil(torch.log2((amax / E4M3_MAX).clamp(min=1e-300)))
                    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
                    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(PAGE_EXP_MIN, PAGE_EXP_MAX).int()
                    r = at % page
                    if r:
                        e = torch.maximum(e, exps[pg])
                        vals[pg][:, :r] = _e4m3(vals[pg][:, :r] * torch.exp2((exps[pg] - e).double())[:, None, None])
                    vals[pg][:, r:r + end - at] = _e4m3(rows * torch.exp2(-e.double())[:, None, None])
                    exps[pg] = e
                    at = end
            back.append((vals, (exps + 127).to(torch.uint8)))
        return q, back[0][0], back[1][0], back[0][1], back[1][1]
    table = s["table"].long()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    for b, (n, t) in enumerate(lens):
        if n == 0:
            continue
        pg = table[b, :-(-t // page)]
        for h in range(H):
            k, v = ((c[pg, h].double() * torch.exp2(sc[pg, h].double() - 127)[:, None, None]).reshape(-1, D)[:t]
                    for c, sc in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            z = torch.einsum("igd,kd->gik", q, k) * s["scale"]
            if case["causal"]:
                z += torch.triu(torch.full((n, t), -math.inf, dtype=torch.float64, device=z.device), diagonal=t - n + 1)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("gik,kd->igd", torch.softmax(z, -1), v)
            lse[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.logsumexp(z, -1).t()
    return out, lse
