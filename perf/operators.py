"""Cases and plain forms of the decode-step operators over an MLA latent cache.

Three operators, in the order a serving step runs them on a layer:

  rope     rotary positions on the RoPE columns of the queries (and their
           gradient): interleaved or half layout, part of a wider head, the
           frequencies plain, linearly interpolated or YaRN-scaled
  append   new tokens' latent rows into a paged cache: the 512 NoPE columns as
           they are, the RoPE columns rotated, as bf16 rows or as FP8 rows
           (512 e4m3 codes, 4 fp32 block scales, bf16 RoPE columns)
  decode   attention of one new token per request over that cache, the whole
           context or the token's own top-k positions

``run`` computes them in elementary torch operations where ``own`` is false
and calls the library where it is true.  ``exact`` is the same result in 64
bits, written from the definitions alone.
"""
import math

import torch

own = False

D_NOPE = 512
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(name, T, H, layout="interleaved", scaling="none", factor=1.0, dtype="bf16", gradient=False, far=1 << 15,
          d_rope=64, head=192):
    return dict(name=name, op="rope", T=T, H=H, layout=layout, scaling=scaling, factor=factor, dtype=dtype,
                gradient=gradient, far=far, d_rope=d_rope, head=head)


def _append(name, requests, new, context, page, fmt="bf16", layout="interleaved", scaling="none", factor=1.0, pad=0,
            d_rope=64):
    return dict(name=name, op="append", requests=requests, new=new, context=context, page=page, fmt=fmt,
                layout=layout, scaling=scaling, factor=factor, pad=pad, d_rope=d_rope)


def _decode(name, B, H, shortest, longest, page=64, fmt="bf16", k=0, d_rope=64):
    return dict(name=name, op="decode", B=B, H=H, shortest=shortest, longest=longest, page=page, fmt=fmt, k=k,
                d_rope=d_rope)


def listed():
    return [
        # one new token's queries of one sequence: the smallest call, latency only
        _rope("rope 1 token, 16 heads", 1, 16),
        # a whole prompt's queries at 32 heads, YaRN-scaled for a long context
        _rope("rope 16384 tokens, YaRN", 16384, 32, scaling="yarn", factor=40.0, far=163840),
        # the gradient in fp32, half layout, 64 rotary columns of a 256-wide head, odd token count
        _rope("rope gradient 8191 tokens", 8191, 16, layout="half", scaling="linear", factor=4.0, dtype="f32",
              gradient=True, head=256),
        # one new token of each of 128 running requests
        _append("append 128 requests", 128, 1, 120, 64),
        # prompt chunks of 8 requests into an FP8 cache, read back as the bf16 rows it stands for
        _append("append 16384 rows, FP8", 8, 2048, 0, 64, fmt="fp8", scaling="yarn", factor=40.0),
        # ragged chunks behind a context, small pages, and the padding tokens of a fixed-size batch
        _append("append ragged, padded", 7, 1171, 333, 16, layout="half", pad=115),
        # one short conversation: latency only
        _decode("decode 1 x 777", 1, 16, 777, 777),
        # one very long context: the length axis is all there is to split
        _decode("decode 1 x 131072", 1, 32, 131072, 131072),
        # a serving batch, ragged over a factor of 64
        _decode("decode 64 x 256..16384", 64, 32, 256, 16384),
        # the same kind of batch over FP8 rows
        _decode("decode 48 x 1024..16384, FP8", 48, 16, 1024, 16384, fmt="fp8"),
        # every head on one GPU, small pages
        _decode("decode 16 x 500..9001, 128 heads", 16, 128, 500, 9001, page=16),
        # the sparse form: each token's own top-2048 positions of a 32k context
        _decode("decode 96 x top-2048 of 32768", 96, 32, 4096, 32768, k=2048),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode"])
    layout = rng.choice(["interleaved", "half"])
    scaling = rng.choice(["none", "linear", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 40.0])
    if op == "rope":
        H = rng.choice([1, 8, 16, 24, 32, 64, 128])
        T = _log(rng, 1, min(16384, 16384 * 32 // H))
        d_rope = rng.choice([32, 64, 64, 128])
        c = _rope("", T, H, layout, scaling, factor, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.4,
                  _log(rng, 4096, 1 << 20), d_rope, d_rope + rng.choice([0, 64, 128, 192]))
        if c["T"] * c["H"] * c["d_rope"] * (2 if c["dtype"] == "f32" else 1) > 16384 * 32 * 64:
            c["T"] = max(1, c["T"] // 4)
    elif op == "append":
        requests = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 16384 // requests))
        page = rng.choice([1, 16, 24, 64, 128])
        c = _append("", requests, new, rng.randrange(0, 300), page, rng.choice(["bf16", "fp8"]), layout, scaling,
                    factor, rng.choice([0, 0, 1, 9]), rng.choice([64, 64, 0]))
    else:
        H = rng.choice([8, 16, 16, 24, 32, 32, 64, 128])
        B = _log(rng, 1, 96)
        most = max(64, min(131072, 250000 * 32 // (max(H, 32) * B)))
        longest = _log(rng, 64, most)
        shortest = max(1, longest // rng.choice([1, 2, 8, 64]))
        k = rng.choice([0, 0, 0, 2048, 100])
        c = _decode("", B, H, shortest, longest, rng.choice([16, 24, 64, 64, 128]), rng.choice(["bf16", "bf16", "fp8"]),
                    k, rng.choice([64, 64, 64, 0]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n lengths over [lo, hi], evenly on a logarithmic scale: the same ones for every seed."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _row_bytes(c):
    return D_NOPE + 16 + 2 * c["d_rope"] if c["fmt"] == "fp8" else 2 * (D_NOPE + c["d_rope"])


def _cache(c, rows, g):
    """A cache of `rows` latent rows: bf16 [rows, 512 + d_rope], or FP8 rows as bytes."""
    if c["fmt"] == "bf16":
        return torch.randn(rows, D_NOPE + c["d_rope"], generator=g, device=DEV, dtype=torch.bfloat16)
    codes = (torch.randn(rows, D_NOPE, generator=g, device=DEV) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (torch.rand(rows, 4, generator=g, device=DEV) + 0.5) / 120
    pe = torch.randn(rows, c["d_rope"], generator=g, device=DEV, dtype=torch.bfloat16)
    return torch.cat([codes.view(torch.uint8), scales.view(torch.uint8), pe.view(torch.uint8).reshape(rows, -1)], 1)


def _pages(lens, page, g):
    """(block table [requests, blocks], pages in the cache): shuffled pages, a few of them free."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 5
    ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    cols = max(max(need), 1)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    at = first[:, None] + torch.arange(cols, device=DEV)[None]
    used = torch.arange(cols, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    return torch.where(used, ids[at.clamp(max=total - 1)], torch.full_like(ids[:1], -1)).contiguous(), total


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # the rotary columns are the last of each head of a projection's output
        x = torch.randn(c["T"], c["H"], c["head"], generator=g, device=DEV, dtype=dt)
        s["x"] = x[..., c["head"] - c["d_rope"]:]
        # consecutive positions of a sequence somewhere in the context
        start = torch.randint(0, max(1, c["far"] - c["T"]), (1,), generator=g, device=DEV)
        s["positions"] = (start + torch.arange(c["T"], device=DEV)).to(torch.int32)
        # they go into the last columns of the latent queries
        full = torch.zeros(c["T"], c["H"], D_NOPE + c["d_rope"] if not c["gradient"] else c["head"], device=DEV, dtype=dt)
        s["out"] = full[..., full.shape[2] - c["d_rope"]:]
    elif c["op"] == "append":
        R, new = c["requests"], c["new"]
        # request r has a few tokens of context more than the one before it
        context = [c["context"] + (7 * r) % 50 for r in range(R)]
        table, total = _pages([n + new for n in context], c["page"], g)
        s["table"] = table
        s["cache"] = _cache(c, total * c["page"], g)
        T = R * new
        s["c_kv"] = torch.randn(T + c["pad"], D_NOPE, generator=g, device=DEV, dtype=torch.bfloat16)
        s["k_pe"] = torch.randn(T + c["pad"], c["d_rope"], generator=g, device=DEV, dtype=torch.bfloat16)
        req = torch.arange(R, device=DEV).repeat_interleave(new)
        pos = torch.tensor(context, device=DEV)[req] + torch.arange(new, device=DEV).repeat(R)
        padding = torch.full((c["pad"],), -1, device=DEV)
        s["positions"] = torch.cat([pos, padding]).to(torch.int32)
        s["token_req"] = torch.cat([req, padding]).to(torch.int32)
    else:
        B, H = c["B"], c["H"]
        lens = _spread(B, c["shortest"], c["longest"])
        order = torch.randperm(B, generator=g, device=DEV)
        table, total = _pages(lens, c["page"], g)
        s["table"] = table[order].contiguous()
        s["lens"] = torch.tensor(lens, device=DEV)[order].to(torch.int32)
        s["cache"] = _cache(c, total * c["page"], g)
        s["q"] = torch.randn(B, H, D_NOPE + c["d_rope"], generator=g, device=DEV, dtype=torch.bfloat16)
        s["scale"] = 192 ** -0.5
        s["idx"] = None
        if c["k"]:
            # k positions, or all of a shorter context, in no order, the rest -1
            pick = torch.rand(B, c["longest"], generator=g, device=DEV)
            pick.masked_fill_(torch.arange(c["longest"], device=DEV)[None] >= s["lens"][:, None], 2.0)
            top = torch.topk(pick, min(c["k"], c["longest"]), dim=1, largest=False)
            idx = torch.full((B, c["k"]), -1, device=DEV, dtype=torch.int32)
            idx[:, :top.indices.shape[1]] = torch.where(top.values < 1.5, top.indices, -1).to(torch.int32)
            s["idx"] = idx
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
ROPE_BASE, ROPE_LEN, BETA_FAST, BETA_SLOW = 10000.0, 4096, 32.0, 1.0


def _mscale(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


def _angles(c, positions):
    """cos and sin (fp32, scaled) of every position and pair; the angles in 64 bits."""
    d = c["d_rope"]
    i = torch.arange(d // 2, device=positions.device, dtype=torch.float64)
    f = ROPE_BASE ** (-2.0 * i / d)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "yarn":
        low = math.floor(d * math.log(ROPE_LEN / (BETA_FAST * 2 * math.pi)) / (2 * math.log(ROPE_BASE)))
        high = math.ceil(d * math.log(ROPE_LEN / (BETA_SLOW * 2 * math.pi)) / (2 * math.log(ROPE_BASE)))
        low, high = max(low, 0), min(high, d - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
    a = positions.to(torch.float64)[:, None] * f
    return (a.cos() * _mscale(c)).float(), (a.sin() * _mscale(c)).float()


def _rotate(c, x, cos, sin):
    """Rotation of the last dimension's pairs; cos and sin broadcast against them."""
    half = x.shape[-1] // 2
    if c["layout"] == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _values(c, rows):
    """The fp32 values of cache rows (the bf16 numbers that an FP8 row stands for)."""
    if c["fmt"] == "bf16":
        return rows.float()
    codes = rows[..., :D_NOPE].contiguous().view(torch.float8_e4m3fn).float()
    scales = rows[..., D_NOPE:D_NOPE + 16].contiguous().view(torch.float32)
    nope = (codes.unflatten(-1, (4, 128)) * scales[..., None]).flatten(-2).bfloat16().float()
    return torch.cat([nope, rows[..., D_NOPE + 16:].contiguous().view(torch.bfloat16).float()], -1)


def _plain_append(s):
    c = s["case"]
    cache, page = s["cache"], c["page"]
    n = c["requests"] * c["new"]  # the padding tokens behind them go nowhere
    pos, req = s["positions"][:n].long(), s["token_req"][:n].long()
    rows = s["table"][req, pos // page].long() * page + pos % page
    pe = s["k_pe"][:n]
    if c["d_rope"]:
        cos, sin = _angles(c, pos)
        pe = _rotate(c, pe.float(), cos, sin).bfloat16()
    if c["fmt"] == "bf16":
        cache[rows] = torch.cat([s["c_kv"][:n], pe], 1)
        return cache
    x = s["c_kv"][:n].float().unflatten(1, (4, 128))
    amax = x.abs().amax(2)
    scales = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    codes = (x / scales[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).flatten(1)
    cache[rows] = torch.cat([codes.view(torch.uint8), scales.view(torch.uint8), pe.contiguous().view(torch.uint8).reshape(n, -1)], 1)
    return _values(c, cache).bfloat16()


def _plain_decode(s):
    c = s["case"]
    page = c["page"]
    if s["idx"] is None:
        pos = torch.arange(c["longest"], device=DEV)[None].expand(c["B"], -1)
        there = pos < s["lens"][:, None]
    else:
        pos, there = s["idx"].long(), s["idx"] >= 0
    pos = torch.where(there, pos, 0)
    rows = s["table"].gather(1, pos // page).long() * page + pos % page
    kv = _values(c, s["cache"][rows])
    score = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
    score = score.masked_fill(~there[:, None], -math.inf)
    top = score.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, kv[..., :D_NOPE]) / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.bfloat16(), "lse": (top + torch.log(total))[..., 0]}


def run(state):
    s, c = state, state["case"]
    if own:
        import dsa_sparse_mla_prefill_gb300 as dsa
        if c["op"] == "decode":
            out, lse = dsa.dsa_paged_decode(s["q"], s["cache"], s["table"], s["lens"], c["page"], s["scale"],
                                            idx=s["idx"])
            return {"out": out, "lse": lse}
        freqs = dsa.dsa_rope_freqs(c["d_rope"], base=ROPE_BASE, layout=c["layout"], scaling=c["scaling"],
                                   factor=c["factor"], original_len=ROPE_LEN, beta_fast=BETA_FAST,
                                   beta_slow=BETA_SLOW, mscale=_mscale(c)) if c["d_rope"] else None
        if c["op"] == "rope":
            return dsa.dsa_rope(s["x"], s["positions"], freqs, out=s["out"], gradient=c["gradient"])
        one_each = c["new"] == 1 and c["pad"] == 0
        cache = dsa.dsa_kv_append(s["c_kv"], s["k_pe"], s["positions"], s["table"], c["page"], s["cache"], rope=freqs,
                                  token_req=None if one_each else s["token_req"])
        return cache if c["fmt"] == "bf16" else dsa.dsa_kv_fp8_dequantize(cache, c["d_rope"])
    if c["op"] == "decode":
        return _plain_decode(s)
    if c["op"] == "append":
        return _plain_append(s)
    cos, sin = _angles(c, s["positions"])
    sign = -1.0 if c["gradient"] else 1.0
    s["out"].copy_(_rotate(c, s["x"].float(), cos[:, None], sign * sin[:, None]))
    return s["out"]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["d_rope"]
        return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["T"], "flops": 3 * n}
    d = D_NOPE + c["d_rope"]
    if c["op"] == "append":
        T = c["requests"] * c["new"]
        b = T * (2 * d + 8 + _row_bytes(c))
        if c["fmt"] == "fp8":  # the rows read back: what the cache holds, as bf16
            rows = (sum(-(-(c["context"] + (7 * r) % 50 + c["new"]) // c["page"]) for r in range(c["requests"])) + 5) * c["page"]
            b += rows * (_row_bytes(c) + 2 * d)
        return {"bytes": b, "flops": T * (3 * c["d_rope"] + (2 * D_NOPE if c["fmt"] == "fp8" else 0))}
    lens = _spread(c["B"], c["shortest"], c["longest"])
    rows = sum(min(n, c["k"]) if c["k"] else n for n in lens)
    table = 4 * (c["B"] * c["k"] if c["k"] else sum(-(-n // c["page"]) for n in lens))
    b = rows * _row_bytes(c) + table + c["B"] * (4 + c["H"] * (2 * d + 2 * D_NOPE + 4))
    return {"bytes": b, "flops": 2 * rows * c["H"] * (d + D_NOPE)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _turned(c, x, positions, back=False):
    """x [tokens, ..., d] with pair i of token t turned by positions[t] * f_i (as complex numbers)."""
    d = c["d_rope"]
    f = []
    for i in range(d // 2):
        w = math.exp(-math.log(ROPE_BASE) * 2 * i / d)
        if c["scaling"] == "linear":
            w /= c["factor"]
        if c["scaling"] == "yarn":
            # pairs that turn more than BETA_FAST times over the first length keep their speed, those that
            # turn less than BETA_SLOW times are slowed down, and those between are mixed
            pair = [d * math.log(ROPE_LEN / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE)) for turns in (BETA_FAST, BETA_SLOW)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), d - 1)
            slow = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w = w * (1 - slow) + w / c["factor"] * slow
        f.append(w)
    a = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(a, 1.0 if c["scaling"] != "yarn" else 1.0 + 0.1 * math.log(c["factor"])), -a if back else a)
    turn = turn.reshape(len(positions), *([1] * (x.dim() - 2)), d // 2)
    x = x.double()
    z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) if c["layout"] == "interleaved" else torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous())
    z = z * turn
    if c["layout"] == "interleaved":
        return torch.view_as_real(z).flatten(-2)
    return torch.cat([z.real, z.imag], -1)


def _wide(c, rows):
    """Cache rows in 64 bits."""
    if c["fmt"] == "bf16":
        return rows.double()
    n = rows.shape[0]
    block = rows[:, 512:528].contiguous().view(torch.float32).double()
    nope = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double().reshape(n, 4, 128) * block[:, :, None]
    nope = nope.reshape(n, 512).float().bfloat16().double()
    if c["d_rope"] == 0:
        return nope
    return torch.cat([nope, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        return _turned(c, s["x"], s["positions"], c["gradient"])
    page, table = c["page"], s["table"].long()
    if c["op"] == "append":
        held = _wide(c, s["cache"])
        n = c["requests"] * c["new"]
        pos, req = s["positions"][:n].long(), s["token_req"][:n].long()
        at = page * table[req, pos // page] + pos % page
        nope = s["c_kv"][:n].double()
        if c["fmt"] == "fp8":
            unit = nope.reshape(n, 4, 128).abs().amax(2, keepdim=True) / 448
            unit = torch.where(unit > 0, unit, torch.ones_like(unit)).float().double()
            code = (nope.reshape(n, 4, 128) / unit).float().to(torch.float8_e4m3fn).double()
            nope = (code * unit).reshape(n, 512)
        held[at, :512] = nope
        if c["d_rope"]:
            held[at, 512:] = _turned(c, s["k_pe"][:n], pos)
        return held
    out = torch.zeros(c["B"], c["H"], 512, dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        pos = torch.arange(int(s["lens"][b]), device=DEV) if s["idx"] is None else s["idx"][b][s["idx"][b] >= 0].long()
        if len(pos) == 0:
            continue
        kv = _wide(c, s["cache"][page * table[b][pos // page] + pos % page])
        score = s["scale"] * (s["q"][b].double() @ kv.T)
        lse[b] = torch.logsumexp(score, 1)
        out[b] = torch.softmax(score, 1) @ kv[:, :512]
    return {"out": out, "lse": lse}
