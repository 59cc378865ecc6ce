"""Plain 64-bit forms of the serving operators, and their error bounds."""
import math

import torch

F64 = torch.float64


def pow2(n):
    """2^n in fp64 by its bits (the device's pow need not be exact)."""
    return ((n + 1023) << 52).view(F64)


def attention(q, k, v, causal, scale):
    """One sequence: q [Lq, Hq, d] over k, v [Lk, Hkv, d].  Returns O, LSE [Hq, Lq], A = sum_j w_j |v_j| and
    B = the largest sum_d |q_d k_d| * |scale| of each row's visible scores."""
    Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[:2]
    g = Hq // Hkv
    q, k, v = q.to(F64), k.to(F64).repeat_interleave(g, 1), v.to(F64).repeat_interleave(g, 1)
    seen = torch.ones(Lq, Lk, dtype=torch.bool, device=q.device)
    if causal:
        i, j = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
        seen = j[None, :] <= (i[:, None] + Lk - Lq)
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    s = torch.where(seen, s, -math.inf)
    if Lk == 0:
        z = torch.zeros(Lq, Hq, d, dtype=F64, device=q.device)
        return z, torch.full((Hq, Lq), -math.inf, dtype=F64, device=q.device), z, z[..., 0].t()
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    e = torch.where(seen, e, 0.0)
    t = e.sum(-1, keepdim=True)
    w = e / torch.where(t == 0, 1.0, t)
    lse = (torch.where(t == 0, -math.inf, m + torch.log(torch.where(t == 0, 1.0, t)))).squeeze(-1)
    b = torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) * abs(scale)
    b = torch.where(seen, b, 0.0).amax(-1)
    return (torch.einsum("hij,jhd->ihd", w, v), lse, torch.einsum("hij,jhd->ihd", w, v.abs()), b)


def check_attention(o, lse, ref, d):
    """Against the 64-bit form, element by element.  What separates them:
    * each score's fp32 sum of d products: at most (d + 2) 2^-24 B, doubled for the reference's own score in
      the exponent; as a relative error of the weights at most e = 2 (d + 3) 2^-24 B + 1.1e-4 (the software
      exponential's 1.01e-4, or the hardware's 2^-22, and fp32 sums);
    * weights rounded to bf16: 2^-8 relative (half a step is eps / 2 = 2^-8 of the value at most);
    * the output's own rounding to bf16: 2^-8 relative, and fp32 accumulation 2^-20 A.
    LSE: the score's error and that of the sum, plus fp32 rounding of the result."""
    o_ref, lse_ref, A, B = ref
    e = 2 * (d + 3) * 2.0 ** -24 * B + 1.1e-4
    eo = e.t().unsqueeze(-1)
    bound = (2.0 ** -8 + 2 * eo + 2.0 ** -20) * A * (1 + 2.0 ** -8) + 2.0 ** -8 * o_ref.abs() + 1e-30
    err = (o.to(F64) - o_ref).abs()
    assert bool((err <= bound).all()), f"|dO| {err.max().item():.3g}, worst {(err / bound).max().item():.3g} of the bound"
    # errors of many roundings average out: a lost bit or a biased rounding would double the mean
    if err.numel() > 4096:
        assert err.mean() <= 0.5 * bound.mean()
    if lse is not None:
        empty = lse_ref == -math.inf
        assert torch.equal(lse.to(F64) == -math.inf, empty)
        d_l = (lse.to(F64) - lse_ref).abs()[~empty]
        b_l = (e + 2.0 ** -23 * (1 + lse_ref.abs()))[~empty]
        assert bool((d_l <= b_l).all()), f"|dLSE| {d_l.max().item():.3g}"
        zero = empty.t().unsqueeze(-1).expand_as(o)
        assert bool((o[zero] == 0).all())


def norm_rope(x, w, eps, pos, freqs, rot, interleaved, amplitude):
    x = x.to(F64)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    if rot == 0:
        return x
    a = pos.to(F64)[:, None, None] * freqs
    c, s = a.cos() * amplitude, a.sin() * amplitude
    y = x.clone()
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def quantise(x):
    """(code values, exponent bytes) of rows in fp64: the smallest 2^e with amax <= 448 * 2^e, e >= -118."""
    x = x.to(F64)
    a = x.abs().amax(-1)
    e = torch.full(a.shape, -118, dtype=torch.int64, device=x.device)
    for n in range(-118, 121):
        e = torch.where(a > 448.0 * 2.0 ** n, n + 1, e)
    e = torch.where(a == 0, 0, e)
    y = x * pow2(-e).unsqueeze(-1)
    m, k = torch.frexp(y.abs().clamp(min=2.0 ** -6))
    step = pow2((k - 1).long() - 3)
    return torch.round(y / step) * step, e + 127


def make_cache(ea, lens, page, Hkv, d, e4m3, seed, width=None, fill=float("nan")):
    """A cache holding random keys and values of the given lengths on shuffled pages; what no sequence wrote is
    `fill` (codes 0x7F and exponent 255 for e4m3).  Returns (KVCache, table, [k], [v] per sequence in bf16)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    perm = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1) if width is None else width), -7, dtype=torch.int32, device="cuda")
    shape = (n_pages, page, Hkv, d)
    ks, vs, at = [], [], 0
    if e4m3:
        pages = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        exps = [torch.full(shape[:3], 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    else:
        pages = [torch.full(shape, fill, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        exps = [None, None]
    for s, n in enumerate(lens):
        ids = perm[at:at + need[s]]
        at += need[s]
        table[s, :need[s]] = ids
        for x, out in ((0, ks), (1, vs)):
            if e4m3:
                c = torch.randint(0, 256, (n, Hkv, d), device="cuda", generator=g).to(torch.uint8)
                c = torch.where((c & 0x7F) == 0x7F, 0x3A, c).to(torch.uint8)
                e = torch.randint(118, 121, (n, Hkv), device="cuda", generator=g).to(torch.uint8)
                val = c.view(torch.float8_e4m3fn).to(F64) * pow2(e.long() - 127).unsqueeze(-1)
            else:
                c, e = torch.randn(n, Hkv, d, device="cuda", generator=g).to(torch.bfloat16), None
                val = c.to(F64)
            out.append(val)
            i = torch.arange(n, device="cuda")
            pages[x][ids[i // page].long(), i % page] = c
            if e is not None:
                exps[x][ids[i // page].long(), i % page] = e
    return ea.KVCache(pages[0], pages[1], *exps), table, ks, vs


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return i32(*out)


def no_device_error(ea):
    rc, word = ea.attn_get_last_device_error()
    assert rc == 0, (rc, hex(word))
