"""Cases and plain forms of the operators that check drafted tokens over an MLA latent cache.

Four operators, in the order a serving step with speculative decoding runs them on a layer:

  norm      RMS norms of the heads of queries and keys with the rotation of
            their RoPE columns in the same pass; also of latent rows, whose
            512 NoPE columns are normed and whose RoPE columns are turned
  gradient  the gradients of inputs and norm weights of the former, for training
  tree      attention of a tree of drafted tokens per request over the paged
            cache: the context, and of the drafted tokens those that a bit mask
            names (a token's ancestors and itself)
  keep      the accepted path's rows move to the positions behind the context,
            in the cache of every layer, and the lengths follow

``run`` computes them in elementary torch operations where ``own`` is false
and calls the library where it is true.  ``exact`` is the same result in 64
bits, written from the definitions alone.
"""
import math

import torch

own = False

D_NOPE = 512
EPS = 1e-6
BASE, ORIGINAL_LEN, BETA_FAST, BETA_SLOW = 10000.0, 4096, 32.0, 1.0
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, T, Hq, Hk, d, d_rope, d_norm=0, layout="interleaved", factor=1.0, dtype="bf16", gradient=False):
    return dict(name=name, op="norm", T=T, Hq=Hq, Hk=Hk, d=d, d_rope=d_rope, d_norm=d_norm or d, layout=layout,
                factor=factor, dtype=dtype, gradient=gradient)


def _tree(name, B, n, H, shortest, longest, page=64, fmt="bf16", d_rope=64, ragged=False):
    return dict(name=name, op="tree", B=B, n=n, H=H, shortest=shortest, longest=longest, page=page, fmt=fmt,
                d_rope=d_rope, ragged=ragged)


def _keep(name, layers, B, n, most, context, page=64, fmt="bf16"):
    return dict(name=name, op="keep", layers=layers, B=B, n=n, most=most, context=context, page=page, fmt=fmt)


def listed():
    return [
        # the drafted tokens of one conversation: queries of 16 heads and the latent key's one: latency only
        _norm("norm 8 tokens, 16 + 1 heads of 192", 8, 16, 1, 192, 64),
        # a whole prompt's queries and per-head keys in front of masked attention
        _norm("norm 16384 tokens, 16 + 16 heads of 192", 16384, 16, 16, 192, 64, factor=40.0),
        # a prompt's latent rows on their way into the cache: 512 columns normed, 64 turned; odd token count
        _norm("norm 32767 latent rows", 32767, 1, 0, 576, 64, d_norm=512, layout="half", factor=40.0),
        # training: whole heads turned in halves, fp32, fewer key heads than query heads, odd token count
        _norm("gradient 4095 tokens, 32 + 8 heads of 128, fp32", 4095, 32, 8, 128, 128, layout="half", dtype="f32",
              gradient=True),
        # training: heads without RoPE columns
        _norm("gradient 8192 tokens, 16 + 16 heads of 256", 8192, 16, 16, 256, 0, gradient=True),
        # one short conversation, four drafted tokens: latency only
        _tree("tree 1 x 777, 4 tokens, 16 heads", 1, 4, 16, 777, 777),
        # a serving batch, eight drafted tokens each, some requests with fewer
        _tree("tree 32 x 512..16384, 8 tokens, 16 heads", 32, 8, 16, 512, 16384, ragged=True),
        # one very long context
        _tree("tree 1 x 131072, 8 tokens, 32 heads", 1, 8, 32, 131072, 131072),
        # every head on one GPU
        _tree("tree 8 x 4096..32768, 4 tokens, 128 heads", 8, 4, 128, 4096, 32768),
        # a wider tree over FP8 rows
        _tree("tree 24 x 1024..16384, 16 tokens, 16 heads, FP8", 24, 16, 16, 1024, 16384, fmt="fp8"),
        # one layer's rows after a step of 16 requests
        _keep("keep 1 layer, 16 requests", 1, 16, 8, 4, 100),
        # every layer of a model at once, a batch of 64 requests
        _keep("keep 61 layers, 64 requests", 61, 64, 16, 6, 60, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gradient", "tree", "tree", "keep"])
    if op in ("norm", "gradient"):
        d, d_norm = rng.choice([(64, 64), (128, 128), (192, 192), (192, 128), (256, 256), (576, 512), (576, 576),
                                (512, 512)])
        Hq, Hk = rng.choice([(1, 0), (8, 1), (16, 16), (24, 24), (32, 8), (64, 8), (128, 1)])
        if d > 256:
            Hq, Hk = rng.choice([(1, 0), (1, 1), (4, 0)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 32 * 192 // ((Hq + Hk) * d * (2 if dtype == "f32" else 1) * (2 if op == "gradient" else 1))
        d_rope = rng.choice([0, 64, 64] + ([d] if d <= 256 else []))
        c = _norm("", _log(rng, 1, min(32768, most)), Hq, Hk, d, d_rope, d_norm, rng.choice(["interleaved", "half"]),
                  rng.choice([1.0, 1.0, 4.0, 40.0]), dtype, op == "gradient")
    elif op == "tree":
        H = rng.choice([8, 16, 16, 24, 32, 64, 128])
        n = rng.choice([n for n in (1, 2, 3, 4, 5, 8, 12, 16, 33, 64) if n * H <= 1024])
        B = _log(rng, 1, 48)
        most = max(96, min(131072, 55_000_000 // (max(n * H, 128) * B)))
        longest = _log(rng, 96, most)
        shortest = max(n, longest // rng.choice([1, 2, 8, 64]))
        c = _tree("", B, n, H, shortest, longest, rng.choice([16, 24, 64, 64, 128]), rng.choice(["bf16", "bf16", "fp8"]),
                  rng.choice([64, 64, 64, 0]), rng.random() < 0.5)
    else:
        fmt = rng.choice(["bf16", "bf16", "fp8"])
        n = rng.choice([2, 4, 8, 16, 33, 64])
        c = _keep("", _log(rng, 1, 61) if fmt == "bf16" else 1, _log(rng, 1, 64), n, rng.randint(1, min(n, 12)),
                  rng.randint(1, 90), rng.choice([1, 16, 24, 64]), fmt)
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


def _drafted(c):
    """Drafted tokens of every request: all n, or in a ragged batch fewer for some (down to one)."""
    return [c["n"] if not c["ragged"] or b % 3 else 1 + (c["n"] - 1) // (1 + b % 4) for b in range(c["B"])]


def _row_bytes(c):
    return D_NOPE + 16 + 2 * c["d_rope"] if c["fmt"] == "fp8" else 2 * (D_NOPE + c["d_rope"])


def _rows(rows, fmt, d_rope, g):
    """Latent rows: bf16 [rows, 512 + d_rope], or FP8 rows as bytes."""
    if fmt == "bf16":
        return torch.randn(rows, D_NOPE + d_rope, generator=g, device=DEV, dtype=torch.bfloat16)
    codes = (torch.randn(rows, D_NOPE, generator=g, device=DEV) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (torch.rand(rows, 4, generator=g, device=DEV) + 0.5) / 120
    pe = torch.randn(rows, d_rope, generator=g, device=DEV, dtype=torch.bfloat16)
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


def _bits(visible):
    """bool [..., 64] -> int64 [...]: element j as bit j."""
    weight = torch.ones(64, dtype=torch.int64, device=visible.device) << torch.arange(64, device=visible.device)
    return (visible.long() * weight).sum(-1)


def _trees(B, n, g):
    """Ancestor masks [B, n] of random trees: token j's parent is an earlier token, or the context."""
    parent = (torch.rand(B, n, generator=g, device=DEV) * torch.arange(1, n + 1, device=DEV)).long() - 1
    visible = torch.zeros(B, n, 64, dtype=torch.bool, device=DEV)
    for j in range(n):
        if j:
            above = visible.gather(1, parent[:, j, None, None].clamp(min=0).expand(-1, 1, 64))[:, 0]
            visible[:, j] = above & (parent[:, j, None] >= 0)
        visible[:, j, j] = True
    return _bits(visible)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        for x, H in (("q", c["Hq"]), ("k", c["Hk"])):
            # projections' outputs: of a size that differs from token to token
            size = torch.rand(c["T"], 1, 1, generator=g, device=DEV) * 2 + 0.2
            s[x] = (torch.randn(c["T"], H, c["d"], generator=g, device=DEV) * size).to(dt) if H else None
            s[x + "_weight"] = (1 + 0.2 * torch.randn(c["d_norm"], generator=g, device=DEV)).to(dt) if H else None
            if c["gradient"]:
                s[x + "_grad"] = torch.randn(c["T"], H, c["d"], generator=g, device=DEV, dtype=dt) if H else None
        # consecutive positions of a sequence somewhere in the context
        start = torch.randint(0, 100000, (1,), generator=g, device=DEV)
        s["positions"] = (start + torch.arange(c["T"], device=DEV)).to(torch.int32)
    elif c["op"] == "tree":
        B, n, H = c["B"], c["n"], c["H"]
        lens = _spread(B, c["shortest"], c["longest"])
        order = torch.randperm(B, generator=g, device=DEV)
        table, total = _pages(lens, c["page"], g)
        s["table"] = table[order].contiguous()
        s["lens"] = torch.tensor(lens, device=DEV)[order].to(torch.int32)
        drafted = torch.minimum(torch.tensor(_drafted(c), device=DEV), torch.tensor(lens, device=DEV))
        s["drafted"] = drafted[order].to(torch.int32)
        s["mask"] = _trees(B, n, g)
        s["cache"] = _rows(total * c["page"], c["fmt"], c["d_rope"], g)
        s["q"] = torch.randn(B, n, H, D_NOPE + c["d_rope"], generator=g, device=DEV, dtype=torch.bfloat16)
        s["scale"] = 192 ** -0.5
    else:
        B, n, most = c["B"], c["n"], c["most"]
        lens = [c["context"] + (7 * b) % 40 + n for b in range(B)]
        s["table"], total = _pages(lens, c["page"], g)
        s["lens"] = torch.tensor(lens, device=DEV).to(torch.int32)
        s["caches"] = [_rows(total * c["page"], c["fmt"], 64, g) for _ in range(c["layers"])]
        # 0 to `most` tokens of each request were accepted.  A path's tokens lie in the order of their depth; one
        # that is not where it belongs already comes from behind the places that are filled.
        behind = torch.rand(B, n - most, generator=g, device=DEV).argsort(1)[:, :most].sort(1).values + most
        stay = torch.randint(0, most + 1, (B, 1), generator=g, device=DEV)
        at = torch.arange(most, device=DEV)[None].expand(B, -1)
        path = at
        if behind.shape[1]:
            path = torch.where(at < stay, at, behind.gather(1, (at - stay).clamp(0, behind.shape[1] - 1)))
        number = torch.randint(0, most + 1, (B, 1), generator=g, device=DEV)
        number = torch.minimum(number, stay + behind.shape[1])
        s["keep"] = torch.where(at < number, path, -1).to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _mscale(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["factor"] > 1.0 else 1.0


def _angles(c, positions):
    """cos and sin (fp32, scaled) of every position and pair; the angles in 64 bits."""
    d = c["d_rope"]
    i = torch.arange(d // 2, device=positions.device, dtype=torch.float64)
    f = BASE ** (-2.0 * i / d)
    if c["factor"] > 1.0:
        low = math.floor(d * math.log(ORIGINAL_LEN / (BETA_FAST * 2 * math.pi)) / (2 * math.log(BASE)))
        high = math.ceil(d * math.log(ORIGINAL_LEN / (BETA_SLOW * 2 * math.pi)) / (2 * math.log(BASE)))
        low, high = max(low, 0), min(high, d - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        f = f / c["factor"] * ramp + f * (1 - ramp)
    a = positions.to(torch.float64)[:, None, None] * f
    return (a.cos() * _mscale(c)).float(), (a.sin() * _mscale(c)).float()


def _rotate(c, x, cos, sin):
    half = x.shape[-1] // 2
    if c["layout"] == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_norm(c, x, weight, cos, sin):
    n, r = c["d_norm"], c["d"] - c["d_rope"]
    v = x.float()
    inv = 1.0 / torch.sqrt((v[..., :n] * v[..., :n]).mean(-1, keepdim=True) + EPS)
    y = torch.cat([v[..., :n] * inv * weight.float(), v[..., n:]], -1)
    if c["d_rope"]:
        y = torch.cat([y[..., :r], _rotate(c, y[..., r:], cos, sin)], -1)
    return y.to(x.dtype)


def _plain_gradient(c, grad, x, weight, cos, sin):
    n, r = c["d_norm"], c["d"] - c["d_rope"]
    v, g = x.float(), grad.float()
    if c["d_rope"]:
        g = torch.cat([g[..., :r], _rotate(c, g[..., r:], cos, -sin)], -1)
    inv = 1.0 / torch.sqrt((v[..., :n] * v[..., :n]).mean(-1, keepdim=True) + EPS)
    unit = v[..., :n] * inv
    gw = g[..., :n] * weight.float()
    gx = inv * (gw - unit * (gw * unit).mean(-1, keepdim=True))
    return torch.cat([gx, g[..., n:]], -1).to(x.dtype), (g[..., :n] * unit).sum((0, 1))


def _values(fmt, rows):
    """The fp32 values of cache rows (the bf16 numbers that an FP8 row stands for)."""
    if fmt == "bf16":
        return rows.float()
    codes = rows[..., :D_NOPE].contiguous().view(torch.float8_e4m3fn).float()
    scales = rows[..., D_NOPE:D_NOPE + 16].contiguous().view(torch.float32)
    nope = (codes.unflatten(-1, (4, 128)) * scales[..., None]).flatten(-2).bfloat16().float()
    return torch.cat([nope, rows[..., D_NOPE + 16:].contiguous().view(torch.bfloat16).float()], -1)


def _plain_tree(s):
    c = s["case"]
    n, page = c["n"], c["page"]
    pos = torch.arange(c["longest"], device=DEV)[None].expand(c["B"], -1)
    there = pos < s["lens"][:, None]
    at = torch.where(there, pos, 0)
    rows = s["table"].gather(1, at // page).long() * page + at % page
    kv = _values(c["fmt"], s["cache"][rows])
    drafted = (pos - (s["lens"] - s["drafted"])[:, None])[:, None]                      # [B, 1, positions]
    live = torch.arange(n, device=DEV)[None, :, None] < s["drafted"][:, None, None]     # [B, n, 1]
    seen = (drafted < 0) | ((s["mask"][:, :, None] >> drafted.clamp(0, 63)) & 1).bool()
    seen = (seen & there[:, None] & live)[:, :, None]                                   # [B, n, 1, positions]
    score = torch.matmul(s["q"].float().flatten(1, 2), kv.transpose(1, 2)).unflatten(1, (n, c["H"])) * s["scale"]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p.flatten(1, 2), kv[..., :D_NOPE]).unflatten(1, (n, c["H"]))
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    return {"out": out.bfloat16(), "lse": (top + torch.log(total))[..., 0]}


def _plain_keep(s):
    c = s["case"]
    page, keep = c["page"], s["keep"].long()
    there = keep >= 0
    context = (s["lens"] - c["n"]).long()[:, None]
    req = torch.arange(c["B"], device=DEV)[:, None].expand_as(keep)[there]
    rows = []
    for pos in ((context + keep)[there], (context + torch.arange(c["most"], device=DEV)[None])[there]):
        rows.append(s["table"][req, pos // page].long() * page + pos % page)
    for cache in s["caches"]:
        cache[rows[1]] = cache[rows[0]]
    lens = (context[:, 0] + there.sum(1)).to(torch.int32)
    return {"caches": [_shown(c, cache) for cache in s["caches"]], "lens": lens}


def _shown(c, cache):
    return cache if c["fmt"] == "bf16" else _values("fp8", cache).bfloat16()


def _own_norm(s, dsa):
    c = s["case"]
    freqs = dsa.dsa_rope_freqs(c["d_rope"], base=BASE, layout=c["layout"], scaling="yarn" if c["factor"] > 1.0 else "none",
                               factor=c["factor"], original_len=ORIGINAL_LEN, beta_fast=BETA_FAST, beta_slow=BETA_SLOW,
                               mscale=_mscale(c)) if c["d_rope"] else None
    if c["gradient"]:
        gq, gk, gqw, gkw = dsa.dsa_qk_norm_rope_gradient(s["q_grad"], s["k_grad"], s["q"], s["k"], s["q_weight"],
                                                         s["k_weight"], s["positions"], freqs, eps=EPS, d_norm=c["d_norm"])
        return {"q": gq, "k": gk, "q_weight": gqw, "k_weight": gkw}
    q, k = dsa.dsa_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], freqs, eps=EPS,
                                d_norm=c["d_norm"])
    return {"q": q, "k": k}


def run(state):
    s, c = state, state["case"]
    if own:
        import dsa_sparse_mla_prefill_gb300 as dsa
        if c["op"] == "norm":
            out = _own_norm(s, dsa)
            return {name: t for name, t in out.items() if t is not None}
        if c["op"] == "tree":
            out, lse = dsa.dsa_tree_decode(s["q"], s["cache"], s["table"], s["lens"], s["mask"], c["page"], s["scale"],
                                           num_draft=s["drafted"])
            return {"out": out, "lse": lse}
        lens = dsa.dsa_kv_keep(s["caches"], s["table"], s["lens"], s["keep"], c["page"], c["n"])
        shown = s["caches"] if c["fmt"] == "bf16" else [dsa.dsa_kv_fp8_dequantize(x, 64) for x in s["caches"]]
        return {"caches": shown, "lens": lens}
    if c["op"] == "tree":
        return _plain_tree(s)
    if c["op"] == "keep":
        return _plain_keep(s)
    cos, sin = _angles(c, s["positions"]) if c["d_rope"] else (None, None)
    out = {}
    for x in ("q", "k"):
        if s[x] is None:
            continue
        if c["gradient"]:
            out[x], out[x + "_weight"] = _plain_gradient(c, s[x + "_grad"], s[x], s[x + "_weight"], cos, sin)
        else:
            out[x] = _plain_norm(c, s[x], s[x + "_weight"], cos, sin)
    return out


def work(case):
    c = case
    if c["op"] == "norm":
        n, size = c["T"] * (c["Hq"] + c["Hk"]) * c["d"], 2 if c["dtype"] == "bf16" else 4
        heads = (c["Hq"] > 0) + (c["Hk"] > 0)
        weights = heads * c["d_norm"] * size
        if c["gradient"]:
            return {"bytes": 3 * n * size + 4 * c["T"] + weights + heads * c["d_norm"] * 4, "flops": 12 * n}
        return {"bytes": 2 * n * size + 4 * c["T"] + weights, "flops": 5 * n}
    if c["op"] == "tree":
        lens = _spread(c["B"], c["shortest"], c["longest"])
        rows, R = sum(lens), c["n"] * c["H"]
        live = sum(n * m for n, m in zip(lens, _drafted(c))) * c["H"]   # (query row, position) pairs
        d = D_NOPE + c["d_rope"]
        table = 4 * sum(-(-n // c["page"]) for n in lens)
        return {"bytes": rows * _row_bytes(c) + table + c["B"] * (8 + 8 * c["n"] + R * (2 * d + 2 * D_NOPE + 4)),
                "flops": 2 * live * (d + D_NOPE)}
    # about half of `most` tokens of a request are kept, and of those half move
    row = D_NOPE + 16 + 128 if c["fmt"] == "fp8" else 2 * (D_NOPE + 64)
    moved = c["B"] * max(1, c["most"]) / 4
    b = 2 * moved * row * c["layers"] + 4 * c["B"] * (c["most"] + 2)
    if c["fmt"] == "fp8":  # the caches read back: what they hold, as bf16
        lens = [c["context"] + (7 * r) % 40 + c["n"] for r in range(c["B"])]
        b += c["layers"] * (sum(-(-n // c["page"]) for n in lens) + 5) * c["page"] * (row + 1152)
    return {"bytes": int(b), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _turned(c, x, positions, back=False):
    """x [tokens, heads, d] with pair i of token t turned by positions[t] * f_i (as complex numbers)."""
    d = c["d_rope"]
    f = []
    for i in range(d // 2):
        w = math.exp(-math.log(BASE) * 2 * i / d)
        if c["factor"] > 1.0:
            # pairs that turn more than BETA_FAST times over the first length keep their speed, those that
            # turn less than BETA_SLOW times are slowed down, and those between are mixed
            pair = [d * math.log(ORIGINAL_LEN / (turns * 2 * math.pi)) / (2 * math.log(BASE)) for turns in (BETA_FAST, BETA_SLOW)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), d - 1)
            slow = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            w = w * (1 - slow) + w / c["factor"] * slow
        f.append(w)
    a = positions.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    m = 1.0 if c["factor"] <= 1.0 else 1.0 + 0.1 * math.log(c["factor"])
    turn = torch.polar(torch.full_like(a, m), -a if back else a)[:, None]
    if c["layout"] == "interleaved":
        z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) * turn
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_norm(c, s):
    out = {}
    n, tail = c["d_norm"], c["d"] - c["d_rope"]
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x, w = s[name].double(), s[name + "_weight"].double()
        rms = (x[..., :n].pow(2).sum(-1, keepdim=True) / n + EPS).sqrt()
        if not c["gradient"]:
            y = x.clone()
            y[..., :n] = x[..., :n] / rms * w
            if c["d_rope"]:
                y[..., tail:] = _turned(c, y[..., tail:], s["positions"])
            out[name] = y
            continue
        g = s[name + "_grad"].double()
        if c["d_rope"]:
            g = torch.cat([g[..., :tail], _turned(c, g[..., tail:], s["positions"], back=True)], -1)
        # d/dx_c of sum_e g_e w_e x_e / rms:  g_c w_c / rms - x_c / (n rms^3) sum_e g_e w_e x_e
        dot = (g[..., :n] * w * x[..., :n]).sum(-1, keepdim=True)
        out[name + "_weight"] = (g[..., :n] * x[..., :n] / rms).sum(1).sum(0)
        g[..., :n] = g[..., :n] * w / rms - x[..., :n] * dot / (n * rms ** 3)
        out[name] = g
    return out


def _wide(fmt, rows):
    """Cache rows in 64 bits."""
    if fmt == "bf16":
        return rows.double()
    n = rows.shape[0]
    block = rows[:, 512:528].contiguous().view(torch.float32).double()
    nope = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double().reshape(n, 4, 128) * block[:, :, None]
    nope = nope.reshape(n, 512).float().bfloat16().double()
    if rows.shape[1] == 528:
        return nope
    return torch.cat([nope, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    page, table = c["page"], s["table"].long()
    if c["op"] == "keep":
        held = [_wide(c["fmt"], x) for x in s["caches"]]
        lens, keep = s["lens"].tolist(), s["keep"].tolist()
        row = lambda b, p: int(table[b, p // page]) * page + p % page
        table = table.cpu()
        src, dst = [], []
        for b in range(c["B"]):
            start = lens[b] - c["n"]
            path = [e for e in keep[b] if e >= 0]
            src += [row(b, start + e) for e in path]
            dst += [row(b, start + i) for i in range(len(path))]
            lens[b] = start + len(path)
        if src:
            src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
            for x in held:
                x[dst] = x[src]
        return {"caches": held, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    out = torch.zeros(c["B"], c["n"], c["H"], 512, dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["n"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        length, drafted = int(s["lens"][b]), int(s["drafted"][b])
        pos = torch.arange(length, device=DEV)
        kv = _wide(c["fmt"], s["cache"][page * table[b][pos // page] + pos % page])
        for i in range(drafted):
            bits = int(s["mask"][b, i])
            tail = [length - drafted + j for j in range(drafted) if bits >> j & 1]
            use = torch.cat([pos[:length - drafted], torch.tensor(tail, device=DEV, dtype=pos.dtype)])
            if len(use) == 0:
                continue
            score = s["scale"] * (s["q"][b, i].double() @ kv[use].T)
            lse[b, i] = torch.logsumexp(score, 1)
            out[b, i] = torch.softmax(score, 1) @ kv[use, :512]
    return {"out": out, "lse": lse}
