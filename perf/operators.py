"""The serving operators around the attention forward, as cases that can be timed and compared.

Four operators that a serving program calls next to ``attention()``:

* ``qk_norm_rope``   RMS norm of every query and key head and the position rotation, one pass;
* ``kv_write`` / ``kv_read``   new tokens into a paged key/value cache (optionally normed and rotated on
  the way, optionally quantised to E4M3 with one power-of-two scale per token and head), and back;
* ``attention_varlen``   attention over packed prompts of different lengths;
* ``attention_paged``    attention of a chunk of new tokens (one token: decoding) over the paged cache.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) where ``own`` is false,
and through the library's entry points where it is true.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

NORM_EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the prompt of a grouped-head model, q and k read out of the fused projection's output
        dict(name="rope prompt 8192", op="qk_norm_rope", T=8192, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             norm=True, far=0),
        # a short prompt of a multi-head model that rotates half of each head, far into a long context
        dict(name="rope far 257", op="qk_norm_rope", T=257, Hq=12, Hkv=12, d=64, rot=32, interleaved=True, norm=False,
             far=900000),
        # one decoding step of 64 sequences into the quantised cache: the smallest call, latency
        dict(name="write step 64 e4m3", op="kv_write", T=64, Hq=32, Hkv=8, d=128, page=16, dtype="e4m3", rope=True,
             pages=512),
        # a prompt's keys and values into the bf16 cache, rotated on the way
        dict(name="write prompt bf16", op="kv_write", T=4096, Hq=32, Hkv=8, d=128, page=64, dtype="bf16", rope=True,
             pages=100),
        # a prefix of a few requests back out of the bf16 cache
        dict(name="read prefix bf16", op="kv_read", n=5, longest=900, Hkv=12, d=64, page=32, dtype="bf16"),
        # long contexts back out of the quantised cache
        dict(name="read long e4m3", op="kv_read", n=8, longest=16000, Hkv=8, d=128, page=16, dtype="e4m3"),
        # a batch of short prompts, GPT-2's heads
        dict(name="prompts gpt2", op="varlen", n=8, longest=1024, Hq=12, Hkv=12, d=64, causal=True),
        # packed prompts of a grouped-head model, up to 8192 tokens
        dict(name="prompts 8192", op="varlen", n=9, longest=8192, Hq=32, Hkv=8, d=128, causal=True),
        # one user decoding at a short context: latency
        dict(name="decode one", op="paged", n=1, q=1, longest=1023, Hq=32, Hkv=8, d=128, page=16, dtype="bf16"),
        # a decoding batch over the quantised cache
        dict(name="decode 64 e4m3", op="paged", n=64, q=1, longest=8192, Hq=32, Hkv=8, d=128, page=64, dtype="e4m3"),
        # chunks of prompts over what is cached of them
        dict(name="chunk bf16", op="paged", n=4, q=512, longest=12000, Hq=32, Hkv=8, d=128, page=16, dtype="bf16"),
        # the last chunk of a long prompt over the quantised cache
        dict(name="chunk 32768 e4m3", op="paged", n=1, q=2048, longest=32768, Hq=32, Hkv=8, d=128, page=64,
             dtype="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    g = rng.choice([1, 2, 3, 4, 8])
    return dict(Hq=min(Hkv * g, 32) // Hkv * Hkv, Hkv=Hkv, d=d)


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_write", "kv_read", "varlen", "paged", "paged"])
    h = _heads(rng)
    if op == "qk_norm_rope":
        return dict(op=op, T=_log(rng, 1, 8192), rot=16 * rng.randint(0 if h["d"] > 64 else 1, h["d"] // 16),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6, far=rng.choice([0, 0, 5000, 900000]), **h)
    if op == "kv_write":
        # at a prompt's size the quantised write takes keys that are rotated already (the prompt's own
        # attention read them); a step's keys are normed and rotated on the way
        dtype = rng.choice(["bf16", "e4m3"])
        T = _log(rng, 1, 4096)
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, T=T, page=page, dtype=dtype, rope=dtype == "bf16" or T <= 256,
                    pages=-(-T // page) + rng.randint(1, 64), **h)
    if op == "kv_read":
        return dict(op=op, n=rng.randint(1, 12), longest=_log(rng, 1, 12000), Hkv=h["Hkv"], d=h["d"],
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "e4m3"]))
    if op == "varlen":
        return dict(op=op, n=rng.randint(1, 16), longest=_log(rng, 1, 4096), causal=rng.random() < 0.8, **h)
    n, q = rng.choice([(1, 1), (3, 1), (17, 1), (40, 1), (2, 4), (5, 7), (1, 300), (3, 129), (2, 900)])
    return dict(op=op, n=n, q=q, longest=max(q, _log(rng, 16, 12000)), page=rng.choice([16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "e4m3"]), **h)


def _lengths(case):
    """The lengths of a case's sequences: the longest, and shorter ones down to a tenth of it."""
    r = random.Random(case["n"] * 1000003 + case["longest"])
    return [case["longest"]] + [max(1, int(case["longest"] * math.exp(-2.3 * r.random()))) for _ in range(case["n"] - 1)]


def _chunks(case):
    """(new tokens, cached tokens with the new ones) of each sequence of a paged case."""
    r = random.Random(case["q"] * 7919 + case["n"])
    lens = _lengths(case)
    new = [case["q"]] + [max(1, int(case["q"] * r.uniform(0.4, 1.0))) for _ in range(case["n"] - 1)]
    return [min(a, b) for a, b in zip(new, lens)], lens


def _visible(new, lens, causal=True):
    return sum(a * b - a * (a - 1) // 2 if causal else a * b for a, b in zip(new, lens))


# ------------------------------------------------------------------ inputs
def _starts(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def _qkv(case, T, gen):
    """q, k and v as slices of one projection's output [T, Hq + 2 Hkv, d]."""
    Hq, Hkv, d = case.get("Hq", 0), case["Hkv"], case["d"]
    x = torch.randn(T, Hq + 2 * Hkv, d, device="cuda", generator=gen).to(torch.bfloat16)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _rope_inputs(case, gen, rot, norm):
    d = case["d"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    freqs = 500000.0 ** (-2.0 * i / max(rot, 1))  # a long-context base
    w = [(1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(torch.bfloat16) for _ in range(2)]
    return dict(freqs=freqs, rot=rot, interleaved=bool(case.get("interleaved", False)),
                q_weight=w[0] if norm else None, k_weight=w[1] if norm else None)


def _cache(case, lens, gen):
    """A paged cache that holds sequences of the given lengths on shuffled pages, and its page table.  What
    no sequence has written holds NaN, as memory that was never written may."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    live = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    at = 0
    for s, n in enumerate(lens):
        ids = perm[at:at + need[s]]
        table[s, :need[s]] = ids
        at += need[s]
        live[ids.long()] = (torch.arange(need[s] * page, device="cuda") < n).view(need[s], page)
    kv = []
    for _ in range(2):
        x = torch.randn(n_pages, page, Hkv, d, device="cuda", generator=gen)
        if case["dtype"] == "bf16":
            kv.append(torch.where(live[..., None, None], x, torch.nan).to(torch.bfloat16))
            continue
        codes, e = _quantise(x)
        kv.append(torch.where(live[..., None, None], codes.view(torch.uint8), 0x7F).to(torch.uint8)
                  .view(torch.float8_e4m3fn))
        kv.append(e)
    if case["dtype"] == "bf16":
        return dict(k=kv[0], v=kv[1], k_exp=None, v_exp=None), table
    return dict(k=kv[0], v=kv[2], k_exp=kv[1], v_exp=kv[3]), table


def _handles(s):
    """The library's own handles for the tensors of a state, which a program keeps as long as the tensors."""
    if own:
        import exact_attention_140_b200 as ea
        if "cache" in s:
            c = s["cache"]
            s["kv"] = ea.KVCache(c["k"], c["v"], c["k_exp"], c["v_exp"])
        if s.get("rope") is not None:
            r = s["rope"]
            s["rot"] = ea.Rope(freqs=r["freqs"], rot_dim=r["rot"], interleaved=r["interleaved"],
                               q_weight=r["q_weight"], k_weight=r["k_weight"], eps=NORM_EPS)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "qk_norm_rope":
        s["q"], s["k"], _ = _qkv(case, case["T"], gen)
        s["pos"] = torch.arange(case["T"], device="cuda", dtype=torch.int64) + case["far"]
        s["rope"] = _rope_inputs(case, gen, case["rot"], case["norm"])
    elif op == "kv_write":
        T, page = case["T"], case["page"]
        s["q"], s["k"], s["v"] = _qkv(case, T, gen)
        s["slots"] = torch.randperm(case["pages"] * page, device="cuda", generator=gen)[:T]
        s["pos"] = torch.randint(0, 32768, (T,), device="cuda", generator=gen)
        s["rope"] = _rope_inputs(case, gen, case["d"], True) if case["rope"] else None
        old = [torch.randn(case["pages"], page, case["Hkv"], case["d"], device="cuda", generator=gen) for _ in range(2)]
        if case["dtype"] == "bf16":
            s["cache"] = dict(k=old[0].to(torch.bfloat16), v=old[1].to(torch.bfloat16), k_exp=None, v_exp=None)
        else:
            (k, ke), (v, ve) = _quantise(old[0]), _quantise(old[1])
            s["cache"] = dict(k=k, v=v, k_exp=ke, v_exp=ve)
    elif op == "kv_read":
        s["lens"] = _lengths(case)
        s["cache"], s["table"] = _cache(case, s["lens"], gen)
        s["cu"] = _starts(s["lens"])
    elif op == "varlen":
        s["lens"] = _lengths(case)
        s["q"], s["k"], s["v"] = _qkv(case, sum(s["lens"]), gen)
        s["cu"] = _starts(s["lens"])
    else:
        s["new"], s["lens"] = _chunks(case)
        s["cache"], s["table"] = _cache(case, s["lens"], gen)
        s["q"] = torch.randn(sum(s["new"]), case["Hq"], case["d"], device="cuda", generator=gen).to(torch.bfloat16)
        s["cu"] = _starts(s["new"])
        s["kv_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    return _handles(s)


# ------------------------------------------------------------------ the operators
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import exact_attention_140_b200 as ea
    case = s["case"]
    op = case["op"]
    if op == "qk_norm_rope":
        return ea.qk_norm_rope(s["q"], s["k"], s["pos"], s["rot"])
    if op == "kv_write":
        c = s["cache"]
        if case["rope"]:
            q = ea.kv_write(s["kv"], s["k"], s["v"], s["slots"], q=s["q"], positions=s["pos"], rope=s["rot"])
        else:
            q = None
            ea.kv_write(s["kv"], s["k"], s["v"], s["slots"])
        return dict(q=q, k=c["k"], v=c["v"], k_exp=c["k_exp"], v_exp=c["v_exp"])
    if op == "kv_read":
        return ea.kv_read(s["kv"], s["table"], s["cu"], sum(s["lens"]))
    if op == "varlen":
        return ea.attention_varlen(s["q"], s["k"], s["v"], s["cu"], s["cu"], causal=case["causal"])
    return ea.attention_paged(s["q"], s["kv"], s["table"], s["kv_lens"], cu_q=s["cu"], max_q=max(s["new"]),
                              causal=True)


def _pow2(k):
    """2^k in float32 for integers k in -126 .. 127, by its bits."""
    return ((k.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., d] as E4M3 codes and one power-of-two exponent per row: value = code * 2^(e - 127) with the
    smallest power that keeps the row's largest magnitude within 448."""
    x = x.float()
    m, k = torch.frexp(x.abs().amax(-1))  # amax = m 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, k - 9, k - 8).clamp(-118, 120)
    k = torch.where(m == 0, 0, k)
    codes = (x * _pow2(-k)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, (k + 127).to(torch.uint8)


def _take(x, at):
    """x[at] for pages of any type (the codes are taken as bytes)."""
    return x[at] if x.dtype == torch.bfloat16 else x.view(torch.uint8)[at].view(x.dtype)


def _dequantise(x, e):
    return x.float() if e is None else x.float() * _pow2(e.int() - 127)[..., None]


def _norm_rope(x, weight, positions, r):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * weight.float()
    rot = r["rot"]
    if rot == 0:
        return x
    angle = positions.double()[:, None] * r["freqs"]  # far positions: the angle in 64 bits
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if r["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _softmax_av(q, k, v, mask, scale):
    """Attention of q [.., Hkv, g, Lq, d] over k, v [.., Hkv, 1, Lk, d], float32: output, log-sum-exp."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    if mask is not None:
        x = x.masked_fill_(~mask, -torch.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -torch.inf, 0.0, m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    return o, (m + total.log()).squeeze(-1)


def _heads_first(q, k, v):
    """[.., L, H, d] tensors as [.., Hkv, g or 1, L, d] in float32."""
    Hkv = k.shape[-2]
    q = q.float().unflatten(-2, (Hkv, q.shape[-2] // Hkv))
    return q.movedim(-4, -2), k.float().movedim(-3, -2).unsqueeze(-3), v.float().movedim(-3, -2).unsqueeze(-3)


def _attend(q, k, v, causal, o, lse):
    """One sequence: q [Lq, Hq, d] over k, v [Lk, Hkv, d] into o and lse."""
    mask = None
    if causal:
        i, j = torch.arange(q.shape[0], device="cuda"), torch.arange(k.shape[0], device="cuda")
        mask = j <= (i + k.shape[0] - q.shape[0])[:, None]
    y, n = _softmax_av(*_heads_first(q, k, v), mask, 1 / math.sqrt(q.shape[-1]))
    o.copy_(y.movedim(-2, 0).reshape(o.shape))
    lse.copy_(n.reshape(lse.shape))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "qk_norm_rope":
        r = s["rope"]
        return (_norm_rope(s["q"], r["q_weight"], s["pos"], r).to(torch.bfloat16),
                _norm_rope(s["k"], r["k_weight"], s["pos"], r).to(torch.bfloat16))
    if op == "kv_write":
        r, c, q, k, v = s["rope"], s["cache"], None, s["k"], s["v"]
        if r is not None:
            q = _norm_rope(s["q"], r["q_weight"], s["pos"], r).to(torch.bfloat16)
            k = _norm_rope(k, r["k_weight"], s["pos"], r)
        for name, x in (("k", k), ("v", v)):
            rows = c[name].flatten(0, 1)
            if c["k_exp"] is None:
                rows[s["slots"]] = x.to(torch.bfloat16)
            else:
                codes, e = _quantise(x)
                rows.view(torch.uint8)[s["slots"]] = codes.view(torch.uint8)
                c[name + "_exp"].flatten(0, 1)[s["slots"]] = e
        return dict(q=q, k=c["k"], v=c["v"], k_exp=c["k_exp"], v_exp=c["v_exp"])
    if op == "varlen":
        o = torch.empty_like(s["q"], memory_format=torch.contiguous_format)
        lse = torch.empty(case["Hq"], o.shape[0], dtype=torch.float32, device="cuda")
        at = 0
        for n in s["lens"]:
            t = slice(at, at + n)
            _attend(s["q"][t], s["k"][t], s["v"][t], case["causal"], o[t], lse[:, t])
            at += n
        return o, lse
    c, page = s["cache"], case["page"]
    if op == "kv_read":
        at = torch.cat([torch.arange(n, device="cuda") for n in s["lens"]])
        seq = torch.repeat_interleave(torch.arange(case["n"], device="cuda"), torch.tensor(s["lens"], device="cuda"))
        ids, row = s["table"][seq, at // page].long(), at % page
        return tuple(_dequantise(_take(c[x], (ids, row)), None if c["k_exp"] is None else c[x + "_exp"][ids, row])
                     .to(torch.bfloat16) for x in ("k", "v"))
    o = torch.empty_like(s["q"])
    lse = torch.empty(case["Hq"], o.shape[0], dtype=torch.float32, device="cuda")

    def rows(name, ids):
        x = _dequantise(_take(c[name], ids), None if c["k_exp"] is None else c[name + "_exp"][ids])
        return x.flatten(-4, -3)

    if max(s["new"]) == 1:  # one token of every sequence: the batch at once
        ids = s["table"].clamp(min=0).long()
        live = torch.arange(ids.shape[1] * page, device="cuda") < s["kv_lens"][:, None]
        k, v = (torch.where(live[..., None, None], rows(x, ids), 0.0) for x in ("k", "v"))
        y, n = _softmax_av(*_heads_first(s["q"][:, None], k, v), live[:, None, None, None], 1 / math.sqrt(case["d"]))
        o.copy_(y.reshape(o.shape))
        lse.copy_(n.reshape(lse.shape[::-1]).t())
        return o, lse
    at = 0
    for i, (a, b) in enumerate(zip(s["new"], s["lens"])):
        t, ids = slice(at, at + a), s["table"][i, :-(-b // page)].long()
        _attend(s["q"][t], rows("k", ids)[:b], rows("v", ids)[:b], True, o[t], lse[:, t])
        at += a
    return o, lse


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    Hq = case.get("Hq", 0)
    cached = d * (2 if case.get("dtype") == "bf16" else 1) + (0 if case.get("dtype") == "bf16" else 1)
    if op == "qk_norm_rope":
        rows = case["T"] * (Hq + Hkv)
        return dict(bytes=rows * d * 4 + case["T"] * 8, flops=rows * d * 8)
    if op == "kv_write":
        T = case["T"]
        rows = T * (2 * Hkv + (Hq if case["rope"] else 0))
        return dict(bytes=rows * d * 2 + T * 16 + 2 * T * Hkv * cached + (T * Hq * d * 2 if case["rope"] else 0),
                    flops=rows * d * 8)
    if op == "kv_read":
        n = 2 * sum(_lengths(case)) * Hkv
        return dict(bytes=n * (cached + 2 * d), flops=n * d)
    if op == "varlen":
        lens = _lengths(case)
        T = sum(lens)
        return dict(bytes=T * (2 * Hq + 2 * Hkv) * d * 2 + T * Hq * 4,
                    flops=4 * Hq * d * _visible(lens, lens, case["causal"]))
    new, lens = _chunks(case)
    return dict(bytes=2 * sum(lens) * Hkv * cached + sum(new) * Hq * (4 * d + 4),
                flops=4 * Hq * d * _visible(new, lens))


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_rope(x, w, pos, r):
    """Each pair (a, b) as the complex number a + ib, turned by e^(i position freq)."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS) * w.double()
    rot = r["rot"]
    if rot == 0:
        return x
    pairs = torch.arange(rot, device="cuda")
    pairs = pairs.view(-1, 2) if r["interleaved"] else pairs.view(2, -1).t()
    z = torch.complex(x[..., pairs[:, 0]], x[..., pairs[:, 1]])
    turn = pos.double()[:, None, None] * r["freqs"].double()
    z = z * torch.polar(torch.ones_like(turn), turn)
    y = x.clone()
    y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """Rows of x rounded to four significant bits (to even; steps of 2^-9 at least) after division by the
    row's power of two: the codes' values."""
    def two_to(n):
        return ((n.long() + 1023) << 52).view(torch.float64)

    top = x.abs().amax(-1, keepdim=True)
    k = torch.full_like(top, -118.0)
    for n in range(-118, 121):  # the powers are tried from the smallest
        k = torch.where(top > 448.0 * 2.0 ** n, n + 1.0, k)
    k = torch.where(top == 0, 0.0, k)
    y = x * two_to(-k)
    step = two_to(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_attention(q, k, v, causal):
    """q [Lq, Hq, d] over k, v [Lk, Hkv, d], one query head at a time."""
    Lq, Hq, d = q.shape
    Lk, g = k.shape[0], Hq // k.shape[1]
    o = torch.zeros(Lq, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((Hq, Lq), -torch.inf, dtype=torch.float64, device="cuda")
    hidden = torch.ones(Lq, Lk, dtype=torch.bool, device="cuda").triu(Lk - Lq + 1) if causal else None
    for h in range(Hq):
        s = q[:, h].double() @ k[:, h // g].double().t() / math.sqrt(d)
        if causal:
            s[hidden] = -torch.inf
        lse[h] = torch.logsumexp(s, -1)
        o[:, h] = torch.exp(s - lse[h][:, None]) @ v[:, h // g].double()
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "qk_norm_rope":
        r = s["rope"]
        return (_exact_rope(s["q"], r["q_weight"], s["pos"], r), _exact_rope(s["k"], r["k_weight"], s["pos"], r))
    if op == "kv_write":
        r, c, q, k, v = s["rope"], s["cache"], None, s["k"].double(), s["v"].double()
        if r is not None:
            q, k = _exact_rope(s["q"], r["q_weight"], s["pos"], r), _exact_rope(k, r["k_weight"], s["pos"], r)
        got = dict(q=q)
        for name, x in (("k", k), ("v", v)):
            got[name] = c[name].double()
            got[name].view(-1, *x.shape[1:])[s["slots"]] = x if c["k_exp"] is None else _exact_e4m3(x)
        return dict(got, k_exp=None, v_exp=None)

    def tokens(name, i, n):
        ids = s["table"][i, :-(-n // case["page"])].long()
        x = _take(s["cache"][name], ids).double()
        if case["dtype"] != "bf16":
            x = x * 2.0 ** (s["cache"][name + "_exp"][ids].double()[..., None] - 127.0)
        return x.flatten(0, 1)[:n]

    if op == "kv_read":
        return tuple(torch.cat([tokens(x, i, n) for i, n in enumerate(s["lens"])]) for x in ("k", "v"))
    if op == "varlen":
        parts, at = [], 0
        for n in s["lens"]:
            t = slice(at, at + n)
            parts.append(_exact_attention(s["q"][t], s["k"][t], s["v"][t], case["causal"]))
            at += n
    else:
        parts, at = [], 0
        for i, (a, b) in enumerate(zip(s["new"], s["lens"])):
            parts.append(_exact_attention(s["q"][at:at + a], tokens("k", i, b), tokens("v", i, b), True))
            at += a
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts], 1)
