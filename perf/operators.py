"""Timed cases of the serving operators: the 8-bit key/value cache (written, read
back, attended to) and decode over a prefix that the whole batch shares.

``own`` selects between the plain form of an operator (elementary torch
operations in 32 bits) and the library's entry points.  Every case is a dict of
plain values; ``prepare`` draws its inputs on the GPU from a seed.

The cache format: a row of D values of one (token, head) is held as D e4m3
codes and one exponent byte e, the smallest e >= 1 with
max |x| <= 448 * 2^(e - 127); the codes are x * 2^(127 - e) rounded to nearest
even, and stand for code * 2^(e - 127).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 8 running sequences: a decode step's cache update (latency)
        dict(name="write_token_b8", op="write", B=8, T=1, N=4096, Hkv=8, D=128, dtype="bf16", ragged=False),
        # a 32K prompt written at the end of its prefill
        dict(name="write_prompt_32k", op="write", B=1, T=32768, N=32896, Hkv=8, D=128, dtype="bf16", ragged=False),
        # right-padded prompts of different lengths (one of them empty), fp32, small heads, odd sizes
        dict(name="write_ragged_fp32", op="write", B=5, T=2049, N=5001, Hkv=2, D=64, dtype="fp32", ragged=True),
        # a short span read back in fp32 (inspection of a cache)
        dict(name="read_span_fp32", op="read", B=2, T=129, N=1000, Hkv=2, D=64, dtype="fp32", ragged=True),
        # contexts read back in bf16, to go on with the dense kernels
        dict(name="read_context_b4", op="read", B=4, T=8191, N=8320, Hkv=8, D=128, dtype="bf16", ragged=True),
        # one short conversation with fp32 queries (latency)
        dict(name="quant_short_fp32", op="quant", B=1, N=257, Hq=8, Hkv=8, D=64, dtype="fp32", ragged=False),
        # a serving batch of mixed lengths
        dict(name="quant_ragged_b16", op="quant", B=16, N=8192, Hq=32, Hkv=8, D=128, dtype="bf16", ragged=True),
        # wide groups (64 query heads over 8), odd cache length
        dict(name="quant_wide_b3", op="quant", B=3, N=20001, Hq=64, Hkv=8, D=128, dtype="bf16", ragged=True),
        # the 128K decode workload: 8 sequences, 32 / 8 heads
        dict(name="quant_128k_b8", op="quant", B=8, N=131072, Hq=32, Hkv=8, D=128, dtype="bf16", ragged=False),
        # two requests behind one system prompt, few heads (latency)
        dict(name="shared_1k_b2", op="shared", B=2, P=1000, N=77, Hq=8, Hkv=2, D=128, dtype="bf16", ragged=True),
        # a serving batch behind one long instruction, its own tails of mixed lengths
        dict(name="shared_8k_b32", op="shared", B=32, P=8192, N=512, Hq=32, Hkv=8, D=128, dtype="bf16", ragged=True),
        # many samples drawn from one 64K document
        dict(name="shared_64k_b128", op="shared", B=128, P=65536, N=256, Hq=32, Hkv=8, D=128, dtype="bf16", ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "quant", "quant", "shared", "shared"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    ragged = rng.random() < 0.6
    if op in ("write", "read"):
        B, T = _log_int(rng, 1, 16), _log_int(rng, 1, 32768)
        while B * T * Hkv * D > 1 << 25:
            B, T = max(1, B // 2), (T if B > 1 else T // 2)
        return dict(op=op, B=B, T=T, N=T + rng.randrange(0, 300), Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    ragged=ragged)
    G = rng.choice([1, 2, 4, 8])
    if op == "quant":
        B, N = _log_int(rng, 1, 32), _log_int(rng, 1, 131072)
        while B * N * Hkv * D > 1 << 29:
            B, N = max(1, B // 2), (N if B > 1 else N // 2)
        return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(["bf16", "bf16", "fp32"]), ragged=ragged)
    B, P, N = _log_int(rng, 1, 128), _log_int(rng, 64, 65536), _log_int(rng, 1, 1024)
    while B * Hkv * G * (P + N) > 1 << 27:
        B, P = max(1, B // 2), (P if B > 1 else P // 2)
    return dict(op=op, B=B, P=P, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, dtype="bf16", ragged=ragged)


def _lengths(B, most, ragged, least):
    """Lengths from `most` down to `least`, fixed by the case: work() counts them too."""
    if not ragged or B == 1:
        return [most] * B
    return [most - (most - least) * i // (B - 1) for i in range(B)]


def _case_lengths(c):
    if c["op"] in ("write", "read"):
        return _lengths(c["B"], c["T"], c["ragged"], 0)
    if c["op"] == "quant":
        return _lengths(c["B"], c["N"], c["ragged"], max(1, c["N"] // 3))
    return _lengths(c["B"], c["N"], c["ragged"], 0)


def work(case):
    c = case
    n, D = sum(_case_lengths(c)), c["D"]
    es = 4 if c["dtype"] == "fp32" else 2
    if c["op"] in ("write", "read"):
        rows = 2 * n * c["Hkv"]
        return {"bytes": rows * (es * D + D + 1), "flops": 3 * rows * D}
    ends = c["B"] * c["Hq"] * (2 * es * D + 4)                       # q, o, lse
    if c["op"] == "quant":
        return {"bytes": 2 * n * c["Hkv"] * (D + 1) + ends, "flops": 4 * n * c["Hq"] * D}
    return {"bytes": 2 * es * (c["P"] + n) * c["Hkv"] * D + ends, "flops": 4 * (c["B"] * c["P"] + n) * c["Hq"] * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(shape, gen, dtype, spread=True):
    """Rows of N(0, 1) values; with `spread`, rows differ in size and a few channels stand out, as keys' do."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if spread:
        x *= 1 + 3 * (torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") ** 4)
        x[..., :: max(1, shape[-1] // 4)] *= 3
    return x.to(dtype)


def _random_cache(B, N, Hkv, D, gen):
    codes, exps = [], []
    for _ in range(2):
        c = torch.empty((B, N, Hkv, D), dtype=torch.float8_e4m3fn, device="cuda")
        e = torch.empty((B, Hkv, N), dtype=torch.uint8, device="cuda")
        for b in range(B):
            c[b], e[b] = _quantise(torch.randn((N, Hkv, D), generator=gen, device="cuda"))
        codes.append(c)
        exps.append(e)
    return codes[0], exps[0], codes[1], exps[1]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, B, D, Hkv = _DT[c["dtype"]], c["B"], c["D"], c["Hkv"]
    lens = _case_lengths(c)
    s = dict(case=c, lens=_int32(lens))
    if c["op"] in ("write", "read"):
        s["cache"] = _random_cache(B, c["N"], Hkv, D, gen)
        # each sequence's span starts behind what its cache already holds
        s["starts"] = _int32([(7 * b + 3) % (c["N"] - c["T"] + 1) for b in range(B)])
        if c["op"] == "write":
            s["k"] = _rows((B, c["T"], Hkv, D), gen, dt)
            s["v"] = _rows((B, c["T"], Hkv, D), gen, dt, spread=False)
        return s
    Hq, G = c["Hq"], c["Hq"] // Hkv
    q = torch.randn((B, Hkv, G, D), generator=gen, device="cuda")
    if c["op"] == "quant":
        s["cache"] = _random_cache(B, c["N"], Hkv, D, gen)
        rows = [torch.randint(0, n, (4,), generator=gen, device="cuda") for n in lens]
        keys = torch.stack([s["cache"][0][b].view(torch.uint8)[r].view(torch.float8_e4m3fn).float() for b, r in enumerate(rows)])
        keys = keys / keys.square().mean(-1, keepdim=True).sqrt().clamp_min(1e-6)
    else:
        s["kp"], s["vp"] = (torch.randn((c["P"], Hkv, D), generator=gen, device="cuda").to(dt) for _ in range(2))
        s["kc"], s["vc"] = (torch.randn((B, c["N"], Hkv, D), generator=gen, device="cuda").to(dt) for _ in range(2))
        keys = s["kp"].float()[torch.randint(0, c["P"], (B, 4), generator=gen, device="cuda")]
    # each query leans towards four keys of its context, planted as in the library's decode workload
    q = q + 6.0 * keys.mean(1)[:, :, None]
    s["q"] = q.reshape(B, Hq, D).to(dt)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _two_to(byte):
    """2^(byte - 127) in fp32, for bytes from 1 to 254: the byte is the number's exponent field."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """x [..., T, H, D] -> codes of the same shape, exponent bytes [..., H, T]."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))                     # max = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    byte = torch.where(m > 0, e + (m > 0.875) - 9 + 127, 1).clamp_min(1)
    codes = (x * _two_to(254 - byte).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, byte.to(torch.uint8).transpose(-1, -2)


def _values(codes, exps):
    return codes.float() * _two_to(exps.transpose(-1, -2)).unsqueeze(-1)


def _span(s):
    """(sequence, token) of every cache row of the call's spans, and the row of the call's own tensors."""
    c = s["case"]
    at = torch.arange(c["T"], device="cuda")
    b, t = torch.nonzero(at[None] < s["lens"][:, None], as_tuple=True)
    return b, t, s["starts"].long()[b] + t


def _attend(q, parts):
    """q [B, Hkv, G, D] against the parts' (scores [B, Hkv, G, n], values, how to multiply): o, lse."""
    scores = torch.cat([p[0] for p in parts], -1)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    z = p.sum(-1, keepdim=True)
    at, o = 0, 0
    for sc, v, how in parts:
        n = sc.shape[-1]
        o = o + torch.einsum(how, p[..., at:at + n], v)
        at += n
    return o / z, (m + torch.log(z)).squeeze(-1)


def _plain(s):
    c = s["case"]
    dt, B, D, Hkv = _DT[c["dtype"]], c["B"], c["D"], c["Hkv"]
    if c["op"] == "write":
        kc, ke, vc, ve = s["cache"]
        b, t, n = _span(s)
        for x, codes, exps in ((s["k"], kc, ke), (s["v"], vc, ve)):
            new, e = _quantise(x)
            codes.view(torch.uint8)[b, n] = new.view(torch.uint8)[b, t]
            exps[b, :, n] = e.transpose(1, 2)[b, t]
        return s["cache"]
    if c["op"] == "read":
        kc, ke, vc, ve = s["cache"]
        b, t, n = _span(s)
        out = []
        for codes, exps in ((kc, ke), (vc, ve)):
            x = torch.zeros((B, c["T"], Hkv, D), dtype=dt, device="cuda")
            rows = codes.view(torch.uint8)[b, n].view(torch.float8_e4m3fn).float()
            x[b, t] = (rows * _two_to(exps[b, :, n]).unsqueeze(-1)).to(dt)
            out.append(x)
        return tuple(out)
    Hq = c["Hq"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D) / math.sqrt(D)
    if c["op"] == "quant":
        kc, ke, vc, ve = s["cache"]
        sc = torch.einsum("bhgd,bnhd->bhgn", q, _values(kc, ke))
        dead = torch.arange(c["N"], device="cuda")[None] >= s["lens"][:, None]
        sc = sc.masked_fill(dead[:, None, None], -math.inf)
        o, lse = _attend(q, [(sc, _values(vc, ve), "bhgn,bnhd->bhgd")])
    else:
        sp = torch.einsum("bhgd,nhd->bhgn", q, s["kp"].float())
        ss = torch.einsum("bhgd,bnhd->bhgn", q, s["kc"].float())
        dead = torch.arange(c["N"], device="cuda")[None] >= s["lens"][:, None]
        ss = ss.masked_fill(dead[:, None, None], -math.inf)
        o, lse = _attend(q, [(sp, s["vp"].float(), "bhgn,nhd->bhgd"), (ss, s["vc"].float(), "bhgn,bnhd->bhgd")])
    return o.reshape(B, Hq, D).to(dt), lse.reshape(B, Hq)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return _plain(s)
    from mass_adaptive_sparse_gb300 import api
    c = s["case"]
    lens = s["lens"] if c["ragged"] else None
    if c["op"] == "write":
        api.cache_write(s["k"], s["v"], s["cache"], starts=s["starts"], new_lens=lens)
        return s["cache"]
    if c["op"] == "read":
        B, T, Hkv, D = c["B"], c["T"], c["Hkv"], c["D"]
        out = tuple(torch.zeros((B, T, Hkv, D), dtype=_DT[c["dtype"]], device="cuda") for _ in range(2)) if c["ragged"] else None
        return api.cache_read(s["cache"], T, dtype=_DT[c["dtype"]], starts=s["starts"], lens=lens, out=out)
    if c["op"] == "quant":
        o, lse, _ = api.decode_quant(s["q"], s["cache"], 0.0, cache_lens=lens)
    else:
        o, lse = api.decode_shared(s["q"], s["kp"], s["vp"], s["kc"], s["vc"], suffix_lens=lens)
    return o, lse


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _power(e):
    """2^e in fp64 for whole numbers e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(y):
    """floor(log2 y) of positive normal fp64 numbers."""
    return (y.view(torch.int64) >> 52) - 1023


def _nearest_e4m3(y):
    """The e4m3 value nearest to each y (|y| <= 448), ties to the even mantissa: normal numbers are
    multiples of 2^(floor(log2 |y|) - 3), those below 2^-6 multiples of 2^-9."""
    step = _power(_floor_log2(y.abs().clamp_min(2.0 ** -6)) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    B, D, Hkv, lens = c["B"], c["D"], c["Hkv"], _case_lengths(c)
    starts = s["starts"].tolist() if "starts" in s else None
    if c["op"] == "write":
        out = []
        for x, codes, exps in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
            codes, exps = codes.double(), exps.clone()
            for b, n in enumerate(lens):
                if n == 0:
                    continue
                rows = x[b, :n].double()
                most = rows.abs().amax(-1)
                e = _floor_log2(most.clamp_min(2.0 ** -126)) - 8       # 448 * 2^e is in most's binade or the next
                e = torch.where(most > 448 * _power(e), e + 1, e).clamp_min(-126)
                codes[b, starts[b]:starts[b] + n] = _nearest_e4m3(rows / _power(e).unsqueeze(-1))
                exps[b, :, starts[b]:starts[b] + n] = (e + 127).T.to(torch.uint8)
            out += [codes, exps]
        return tuple(out)
    if c["op"] == "read":
        out = []
        for codes, exps in (s["cache"][:2], s["cache"][2:]):
            x = torch.zeros((B, c["T"], Hkv, D), dtype=torch.float64, device="cuda")
            for b, n in enumerate(lens):
                at = slice(starts[b], starts[b] + n)
                x[b, :n] = codes[b, at].double() * _power(exps[b, :, at].long() - 127).T.unsqueeze(-1)
            out.append(x)
        return tuple(out)
    G = c["Hq"] // Hkv
    o = torch.empty((B, c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, c["Hq"]), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        if c["op"] == "shared":
            kp, vp = s["kp"][:, h].double(), s["vp"][:, h].double()
        for b, n in enumerate(lens):
            if c["op"] == "quant":
                kc, ke, vc, ve = s["cache"]
                k = kc[b, :n, h].double() * _power(ke[b, h, :n].long() - 127)[:, None]
                v = vc[b, :n, h].double() * _power(ve[b, h, :n].long() - 127)[:, None]
            else:
                k, v = torch.cat([kp, s["kc"][b, :n, h].double()]), torch.cat([vp, s["vc"][b, :n, h].double()])
            heads = slice(h * G, (h + 1) * G)
            z = (s["q"][b, heads].double() / math.sqrt(D)) @ k.T
            l = torch.logsumexp(z, -1)
            lse[b, heads] = l
            o[b, heads] = torch.exp(z - l[:, None]) @ v
    return o, lse
