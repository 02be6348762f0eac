"""The decode step on the GPU against the 64-bit oracle: rotary positions and
their gradient, cache append, paged attention of one token per request; edges
of each, streams, captured graphs, and the three run as one step.

Tolerances, from the arithmetic (u = 2^-24, half a step of float32; a bf16
rounding is off by at most 2^-8 of the value):
  rope      the angle is a float32 number of half turns, off by at most 2^-25
            half turns (pi 2^-25 = 1.6 u rad), cos and sin are 2-ulp functions
            scaled once (at most 5 u together), each product and the sum round
            (3 u): at most 10 u of |m| (|a| + |b|) per output, then the bf16
            rounding.
  decode    scores: 576 products summed in float32, each addition off by at
            most one step (2 u) of the sum of magnitudes M: 1152 u M, and 3 u
            for scale and log2(e).  P is rounded to bf16 and divided by the sum
            of the rounded P: every weight is off by at most 2^-8 each way, so
            an output is off by at most 2 (2^-8 + 1155 u M) sum_j w_j |c_j|,
            with 2^-16 of it for the products above one, and its own rounding.
            lse: 1155 u M, exp2 and log2 (2^-21), and the sum's own roundings
            (tiles + 32 additions, u each), and 4 u of |lse|.
"""
import math

import numpy as np
import pytest

import oracle.dsa_oracle as O
from gpu_util import bf, f32, i32, need_gpu, torch
from synth import normal_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _clean():
    import dsa_sparse_mla_prefill_gb300 as dsa
    dsa.dsa_last_device_error()
    yield
    st, counts = dsa.dsa_last_device_error()
    assert st == 0 and counts[1] == 0, counts


def bad_count():
    import dsa_sparse_mla_prefill_gb300 as dsa
    torch.cuda.synchronize()
    st, counts = dsa.dsa_last_device_error()
    assert st == 0, counts
    return counts[0]


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


# ---------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------
def rope_case(seed, T, H, d, dtype, pos_hi, pos_lo=0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, d)).astype(np.float32)
    x = torch.from_numpy(x).to("cuda").to(dtype)
    pos = rng.integers(pos_lo, pos_hi, T).astype(np.int32)
    pos[:1] = pos_hi - 1
    return x, pos


def check_rope(got, x, pos, f, layout, m=1.0, gradient=False):
    xd = x.double().cpu().numpy()
    want = O.rope(xd, pos, f, layout, m, gradient)
    d = xd.shape[-1]
    a, b = (xd[..., 0::2], xd[..., 1::2]) if layout == "interleaved" else (xd[..., :d // 2], xd[..., d // 2:])
    pair = np.abs(a) + np.abs(b)
    pair = np.repeat(pair, 2, axis=-1) if layout == "interleaved" else np.concatenate([pair, pair], -1)
    tol = 10 * U * abs(m) * pair
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,d", [(1, 1, 2), (1, 16, 64), (3, 5, 6), (7, 1, 20), (33, 24, 64), (257, 3, 128), (2, 128, 256)])
@pytest.mark.parametrize("gradient", [False, True])
def test_rope(layout, dtype, T, H, d, gradient):
    import dsa_sparse_mla_prefill_gb300 as dsa
    x, pos = rope_case(T + d, T, H, d, dtype, 200000)
    keep = x.clone()
    fr = dsa.dsa_rope_freqs(d, layout=layout, mscale=1.3)
    got = dsa.dsa_rope(x, i32(pos), fr, gradient=gradient)
    check_rope(got, x, pos, O.rope_frequencies(d, 10000.0), layout, np.float64(np.float32(1.3)), gradient)
    assert torch.equal(x, keep)


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("yarn", 40.0)])
def test_rope_far_positions(scaling, factor):
    import dsa_sparse_mla_prefill_gb300 as dsa
    f = O.rope_frequencies(64, 10000.0, scaling, factor)
    x, pos = rope_case(5, 300, 2, 64, torch.float32, 1 << 20, -(1 << 20))
    fr = dsa.dsa_rope_freqs(64, scaling=scaling, factor=factor)
    check_rope(dsa.dsa_rope(x, i32(pos), fr), x, pos, f, "interleaved")
    # the largest and smallest positions: the table itself is within 2^-51 turns per position of the
    # frequencies, and the 64-bit oracle within p 2^-53 rad of its own, so both add p 2^-49 rad at most
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 0], dtype=np.int32)
    x = x[:4].contiguous()
    got = dsa.dsa_rope(x, i32(pos), fr).double().cpu().numpy()
    want = O.rope(x.double().cpu().numpy(), pos, f, "interleaved")
    xd = np.abs(x.double().cpu().numpy())
    pair = np.repeat(xd[..., 0::2] + xd[..., 1::2], 2, axis=-1)
    assert (np.abs(got - want) <= (10 * U + 2.0 ** (31 - 49)) * pair).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_views(layout, dtype):
    """Part of a wider head, other orders of dimensions, odd offsets, in place, broadcast."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    fr = dsa.dsa_rope_freqs(32, layout=layout)
    f = O.rope_frequencies(32, 10000.0)
    wide, pos = rope_case(9, 19, 6, 100, dtype, 5000)
    p = i32(pos)
    for lo in (0, 8, 3, 68):
        x = wide[..., lo:lo + 32]
        check_rope(dsa.dsa_rope(x, p, fr), x, pos, f, layout)
        dst = torch.full((19, 6, 576), 7.0, dtype=dtype, device="cuda")
        assert dsa.dsa_rope(x, p, fr, out=dst[..., 512:544]).data_ptr() == dst[..., 512:544].data_ptr()
        check_rope(dst[..., 512:544], x, pos, f, layout)
        assert (dst[..., :512] == 7).all() and (dst[..., 544:] == 7).all()
        own = wide.clone()
        dsa.dsa_rope(own[..., lo:lo + 32], p, fr, out=own[..., lo:lo + 32])   # in place
        check_rope(own[..., lo:lo + 32], x, pos, f, layout)
        own[..., lo:lo + 32] = wide[..., lo:lo + 32]
        assert torch.equal(own, wide)
    # heads outside tokens, and a head shared by broadcasting
    hm = wide[..., :32].transpose(0, 1).contiguous().transpose(0, 1)
    check_rope(dsa.dsa_rope(hm, p, fr), hm, pos, f, layout)
    out = torch.empty_like(hm)
    dsa.dsa_rope(hm, p, fr, out=out)
    check_rope(out, hm, pos, f, layout)
    one = wide[:, :1, :32].expand(19, 6, 32)
    check_rope(dsa.dsa_rope(one, p, fr), one, pos, f, layout)


def test_rope_empty_and_refusals():
    import dsa_sparse_mla_prefill_gb300 as dsa
    fr = dsa.dsa_rope_freqs(64)
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert dsa.dsa_rope(x, i32(np.zeros(0)), fr).shape == (0, 4, 64)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = i32(np.zeros(3))
    for bad in (lambda: dsa.dsa_rope(x[..., ::2], pos, dsa.dsa_rope_freqs(32)), lambda: dsa.dsa_rope(x, pos[:2], fr),
                lambda: dsa.dsa_rope(x, pos, dsa.dsa_rope_freqs(32)), lambda: dsa.dsa_rope(x, pos, fr, out=x[:2]),
                lambda: dsa.dsa_rope(x, pos, fr, out=x.float()), lambda: dsa.dsa_rope(x, pos.cpu(), fr)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dsa.DSAError):                                   # overlapping heads of the result
        dsa.dsa_rope(x, pos, fr, out=x[:, :1].expand(3, 4, 64))


def test_rope_gradient_is_the_difference_quotient():
    import dsa_sparse_mla_prefill_gb300 as dsa
    fr = dsa.dsa_rope_freqs(64, mscale=1.1)
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).cuda()
    g = torch.from_numpy(rng.standard_normal((6, 2, 64)).astype(np.float32)).cuda()
    pos = i32(rng.integers(0, 9000, 6))
    dx = dsa.dsa_rope(g, pos, fr, gradient=True)
    # the map is linear, so the difference over a step of one is the directional derivative
    diff = dsa.dsa_rope(x + v, pos, fr).double() - dsa.dsa_rope(x, pos, fr).double()
    lhs, rhs = (diff * g.double()).sum().item(), (v.double() * dx.double()).sum().item()
    # each output within 13 u (10 and the rounding of x + v) of 1.1 (|a| + |b|): a bound on the two sums
    size = 1.1 * 4 * ((x.abs() + v.abs()).double().norm() * g.double().norm()).item()
    assert abs(lhs - rhs) <= 26 * U * size


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def table_of(rng, lens, bs, spare=3, cols=0):
    nb = [-(-n // bs) for n in lens]
    ids = rng.permutation(sum(nb) + spare)
    bt = np.full((len(lens), max(max(nb), 1) + cols), -1, dtype=np.int32)
    p = 0
    for r, n in enumerate(nb):
        bt[r, :n] = ids[p:p + n]
        p += n
    return bt, (sum(nb) + spare) * bs


def check_rows(cache_rows_pe, pe_bits, pos, f, layout, m):
    want = O.rope(O.bf16_to_f64(pe_bits)[:, None], pos, f, layout, m)[:, 0]
    x = np.abs(O.bf16_to_f64(pe_bits))
    d = x.shape[1]
    pair = np.repeat(x[:, 0::2] + x[:, 1::2], 2, axis=1) if layout == "interleaved" else \
        np.tile(x[:, :d // 2] + x[:, d // 2:], (1, 2))
    tol = 10 * U * m * pair
    tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(O.bf16_to_f64(cache_rows_pe) - want) <= tol).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("layout,d_rope,bs", [("interleaved", 64, 64), ("half", 64, 3), ("interleaved", 0, 16)])
@pytest.mark.parametrize("T", [1, 9, 1500])
def test_append(fmt, layout, d_rope, bs, T):
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(T + bs)
    R = 1 if T == 1 else 4
    lens = [T + 40] * R
    bt, N = table_of(rng, lens, bs)
    req = rng.integers(0, R, T).astype(np.int32)
    pos = rng.permutation(T + 40)[:T].astype(np.int32)          # distinct positions: distinct rows
    if T > 1:
        pos[T // 2] = -1                                        # padding
        pos[1] = bt.shape[1] * bs                               # past the table
        pos[3], req[3] = 0, R                                   # no such request
        pos[5] = -7
    c, pe = normal_bf16(rng, (T, 512)), normal_bf16(rng, (T, max(d_rope, 1)))
    c[0, :128] = 0                                              # an all-zero block
    wide = torch.zeros(T, 512 + max(d_rope, 8), dtype=torch.bfloat16, device="cuda")
    wide[:, :512] = bf(c)
    if d_rope:
        wide[:, 512:] = bf(pe)
    fr = dsa.dsa_rope_freqs(64, layout=layout, scaling="yarn", factor=8.0, mscale=1.2) if d_rope else None
    if fmt == "bf16":
        cache = bf(normal_bf16(rng, (N, 512 + d_rope + 8)))
    else:
        cache = torch.from_numpy(rng.integers(0, 255, (N, 528 + 2 * d_rope), dtype=np.uint8)).cuda()
    before = cache.clone()
    rows, bad = O.append_rows(pos, req, bt, bs, N)
    got = dsa.dsa_kv_append(wide[:, :512], wide[:, 512:512 + d_rope] if d_rope else None, i32(pos), i32(bt), bs, cache,
                            rope=fr, token_req=i32(req))
    assert got is cache and bad_count() == bad
    t = np.flatnonzero(rows >= 0)
    r = rows[t]
    untouched = np.setdiff1d(np.arange(N), r)
    assert torch.equal(cache[untouched.tolist()], before[untouched.tolist()])
    if fmt == "bf16":
        host = bits(cache)
        assert np.array_equal(host[r, :512], c[t])
        assert np.array_equal(host[:, 512 + d_rope:], bits(before)[:, 512 + d_rope:])   # columns behind the row
        pe_got = host[r, 512:512 + d_rope]
    else:
        host = cache.cpu().numpy()
        assert np.array_equal(host[r, :528], O.kv_fp8_quantize(c[t], 0))
        pe_got = np.ascontiguousarray(host[r, 528:]).view(np.uint16)
    if d_rope:
        f = O.rope_frequencies(64, 10000.0, "yarn", 8.0)
        check_rows(pe_got, pe[t], pos[t], f, layout, np.float64(np.float32(1.2)))


def test_append_unrotated_and_own_request():
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(2)
    bt, N = table_of(rng, [20, 20, 20], 16)
    c, pe = normal_bf16(rng, (3, 512)), normal_bf16(rng, (3, 64))
    cache = torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda")
    pos = np.array([19, 0, 7], dtype=np.int32)
    dsa.dsa_kv_append(bf(c), bf(pe), i32(pos), i32(bt), 16, cache)
    rows, bad = O.append_rows(pos, None, bt, 16, N)
    assert bad_count() == bad == 0
    assert np.array_equal(bits(cache)[rows], np.concatenate([c, pe], 1))
    # the FP8 row is the quantize kernel's
    f8 = torch.zeros(N, 656, dtype=torch.uint8, device="cuda")
    dsa.dsa_kv_append(bf(c), bf(pe), i32(pos), i32(bt), 16, f8)
    assert torch.equal(f8[rows.tolist()], dsa.dsa_kv_fp8_quantize(cache, 64)[rows.tolist()])
    # nothing to do
    e = torch.zeros(0, 512, dtype=torch.bfloat16, device="cuda")
    dsa.dsa_kv_append(e, e[:, :64], i32(np.zeros(0)), i32(bt), 16, cache)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
class Decode:
    """A batch of requests over a shuffled paged cache whose unnamed rows are NaN."""

    def __init__(self, seed, lens, H, bs=16, d_rope=64, fmt="bf16", k=0, scale=192 ** -0.5, spread=1.0, ld_extra=0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.bs, self.scale, self.fmt = np.asarray(lens, dtype=np.int32), H, bs, scale, fmt
        self.d_qk = 512 + d_rope
        B = len(lens)
        self.bt, self.N = table_of(rng, np.maximum(self.lens, 0), bs)
        self.q = normal_bf16(rng, (B, H, self.d_qk))
        kv = normal_bf16(rng, (self.N, self.d_qk))
        if spread != 1.0:   # scores that range widely
            self.q = O._f32_to_bf16_bits((O.bf16_to_f64(self.q) * spread).astype(np.float32))
        used = np.zeros(self.N, dtype=bool)
        for b, n in enumerate(self.lens):
            for p in range(max(int(n), 0)):
                used[self.bt[b, p // bs] * bs + p % bs] = True
        self.used = used
        if fmt == "bf16":
            kv[~used] = 0x7fc0
            self.cache = torch.full((self.N, self.d_qk + ld_extra), float("nan"), dtype=torch.bfloat16, device="cuda")
            self.cache[:, :self.d_qk] = bf(kv)
            self.values = O.bf16_to_f64(kv)
        else:
            rows = O.kv_fp8_quantize(kv, d_rope)
            self.values = O.bf16_to_f64(O.kv_fp8_dequantize(rows, d_rope))
            rows[~used] = 0x7f                                        # NaN codes, NaN scales, NaN RoPE columns
            self.cache = torch.from_numpy(rows).cuda()
        self.values[~used] = np.nan
        self.k = k
        self.idx = None
        if k:
            self.idx = np.full((B, k + 3), -1, dtype=np.int32)
            for b, n in enumerate(self.lens):
                m = min(k, max(int(n), 0))
                cols = rng.permutation(k)[:m]
                self.idx[b, cols] = rng.permutation(max(int(n), 0))[:m]
                self.idx[b, k:] = 123456789                            # columns behind k are not looked at

    def run(self, **kw):
        import dsa_sparse_mla_prefill_gb300 as dsa
        kw = dict(dict(idx=None if self.idx is None else i32(self.idx), k=self.k or None), **kw)
        return dsa.dsa_paged_decode(bf(self.q), self.cache, i32(self.bt), i32(self.lens), self.bs, self.scale, **kw)

    def check(self, got, bad=0):
        out, lse = got
        ref = O.paged_decode(self.q, self.values, self.bt, self.lens, self.bs, self.scale, self.idx, self.k or None)
        assert bad_count() == ref["bad"] == bad
        M = ref["mass"]
        score = 1155 * U * M
        w = 2 * (2.0 ** -8 + score) * ref["spread"].transpose(2, 0, 1) * (1 + 2.0 ** -7)
        tol = w.transpose(1, 2, 0) + 2.0 ** -8 * np.abs(ref["out"]) + 1e-30
        err = np.abs(f32(out) - ref["out"])
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
        got_l = lse.double().cpu().numpy()
        inf = np.isinf(ref["lse"])
        assert np.array_equal(inf, np.isneginf(got_l))
        tiles = -(-max(int(self.lens.max()), 1) // 128)
        ltol = score + 2.0 ** -21 + (tiles + 32) * U + 4 * U * np.where(inf, 0, np.abs(ref["lse"]))
        lerr = np.abs(np.where(inf, 0, got_l) - np.where(inf, 0, ref["lse"]))
        assert (lerr <= ltol).all(), float((lerr / ltol).max())


FMTS = ["bf16", "fp8"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [1, 16, 32])
@pytest.mark.parametrize("lens", [[1], [0], [128], [129], [2, 0, 127, 0, 0, 300]])
def test_decode_small(fmt, H, lens):
    d = Decode(1, lens, H, fmt=fmt)
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,d_rope,bs", [(8, 64, 1), (16, 0, 7), (24, 64, 24), (32, 0, 64), (33, 64, 100), (64, 64, 128),
                                         (96, 0, 256), (128, 64, 16)])
def test_decode_shapes(fmt, H, d_rope, bs):
    d = Decode(H, [700, 33, 0, 257, 1024, 5], H, bs=bs, d_rope=d_rope, fmt=fmt, ld_extra=8)
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [16, 32, 128])
def test_decode_long_context_is_split(fmt, H):
    d = Decode(7, [20011], H, bs=64, fmt=fmt)
    d.check(d.run())


@pytest.mark.parametrize("H,d_rope,bs,k", [(65, 64, 4, 0), (100, 0, 64, 0), (128, 64, 128, 0), (127, 64, 100, 0),
                                           (80, 64, 16, 300), (128, 0, 64, 77)])
def test_decode_head_pairs(H, d_rope, bs, k):
    """More than 64 heads: two CTAs share every row; heads that fill neither, boxes and gathers mixed in a tile's run,
    requests without keys, ranges without tiles."""
    d = Decode(H, [700, 33, 0, 257, 1024, 5, 0, 128, 2500], H, bs=bs, d_rope=d_rope, k=k, ld_extra=8, spread=3.0)
    d.check(d.run())
    d.lens = np.array([3, 0, 0, 0, 0, 0, 0, 0, 0], np.int32)
    if k:
        d.idx[1:] = -1
        d.idx[0, :k] = -1
        d.idx[0, k - 1] = 2
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_calls_in_a_row_give_the_same_bits(fmt):
    """Launches that overlap each other's ends, of different head counts and in one workspace."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    sets = [Decode(40 + i, [2000, 64, 0, 5000], H, bs=64, fmt=fmt) for i, H in enumerate((16, 128, 32))]
    ws = torch.empty(max(dsa.dsa_paged_decode_workspace(4, d.H, d.bt.shape[1] * 64) for d in sets), dtype=torch.uint8,
                     device="cuda")
    args = [(bf(d.q), d.cache, i32(d.bt), i32(d.lens), 64, d.scale) for d in sets]
    first = [d.run() for d in sets]
    for d, got in zip(sets, first):
        d.check(got)
    outs = [[dsa.dsa_paged_decode(*a, workspace=ws) for a in args] for _ in range(20)]
    torch.cuda.synchronize()
    for row in outs:
        for (o, l), (o0, l0) in zip(row, first):
            assert torch.equal(o, o0) and torch.equal(l, l0)
    assert bad_count() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_many_short_requests(fmt):
    rng = np.random.default_rng(5)
    d = Decode(8, rng.integers(0, 200, 900), 16, fmt=fmt)
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [1, 100, 128, 300])
def test_decode_own_positions(fmt, k):
    d = Decode(9, [1000, 50, 0, 300, 1], 32, fmt=fmt, k=k)
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_wide_scores(fmt):
    """Scores over hundreds of powers of two: the running max moves often, most weights vanish."""
    d = Decode(10, [900, 4000], 32, fmt=fmt, spread=30.0)
    d.check(d.run())


def test_decode_rising_scores():
    """The largest scores come last, in every part of a split context."""
    d = Decode(11, [6000], 16)
    q = O.bf16_to_f64(d.q)[0, 0]
    for p in range(0, 6000, 50):
        r = d.bt[0, p // 16] * 16 + p % 16
        v = O._f32_to_bf16_bits((q * (0.5 + p / 1500.0)).astype(np.float32))
        d.values[r] = O.bf16_to_f64(v)
        d.cache[int(r), :576] = bf(v)
    d.check(d.run())


def test_decode_negative_and_zero_scale():
    for scale in (-0.05, 0.0):
        d = Decode(12, [300, 1, 1300], 16, scale=scale)
        d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_bad_entries_are_absent(fmt):
    d = Decode(13, [200, 90, 64, 500], 16, bs=16, fmt=fmt, k=60)
    # positions outside the request, and lengths
    d.idx[0, 3], d.idx[0, 40], d.idx[1, 7] = 200, -2, 2 ** 31 - 1
    # an unmapped page and one outside the cache
    d.bt[3, 2], d.bt[3, 5] = -4, d.N // 16
    listed = [x for x in d.idx[3, :60] if x // 16 in (2, 5) and x >= 0]
    d.check(d.run(), bad=3 + len(listed))
    # the whole context: the lost pages' positions are counted
    e = Decode(13, [200, 90, 64, 500], 16, bs=16, fmt=fmt)
    e.bt[3, 2], e.bt[3, 5] = -4, e.N // 16
    e.lens[2] = 10 ** 6                                               # cut to the table's width, counted once
    e.bt[2, 4:] = -1
    e.check(e.run(), bad=32 + 1 + (e.bt.shape[1] - 4) * 16)
    # every page lost, no row at all
    e.bt[:] = -1
    e.lens[:] = [3, 0, -5, 1]
    e.check(e.run(), bad=4)


def test_decode_empty_cache():
    import dsa_sparse_mla_prefill_gb300 as dsa
    q = bf(normal_bf16(np.random.default_rng(1), (2, 16, 576)))
    cache = torch.empty(0, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = dsa.dsa_paged_decode(q, cache, i32([[0], [0]]), i32([5, 0]), 16, 1.0)
    assert bad_count() == 5
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = dsa.dsa_paged_decode(q[:0], cache, i32(np.zeros((0, 1))), i32(np.zeros(0)), 16, 1.0)
    assert out.shape == (0, 16, 512)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_same_bits_and_shared_workspace(fmt):
    """The same call twice, in a workspace full of NaN that another shape has used in between."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    d, e = Decode(14, [3000, 777, 129], 32, fmt=fmt), Decode(15, [2500], 32, fmt=fmt)
    ws = torch.full((dsa.dsa_paged_decode_workspace(3, 32, d.bt.shape[1] * 16),), 255, dtype=torch.uint8, device="cuda")
    a = d.run(workspace=ws)
    e.check(e.run(workspace=ws))
    b = d.run(workspace=ws)
    torch.cuda.synchronize()
    assert np.array_equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])
    d.check(b)


def test_decode_on_another_stream_and_outputs_kept():
    """A side stream; rows of the caller's tensors behind the last request stay as they are."""
    d = Decode(16, [500, 1500], 16)
    big = torch.full((4, 16, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 16), 5.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = d.run(out=big[:2], lse=lse[:2], stream=s)
    s.synchronize()
    d.check(got)
    assert (big[2:] == 5).all() and (lse[2:] == 5).all()
    with torch.cuda.stream(s):
        got = d.run()
    s.synchronize()
    d.check(got)


def test_decode_graph_follows_lengths():
    """One captured call, replayed as the lengths, the table and the queries change, beside another
    captured call with its own workspace."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    d = Decode(17, [900, 40, 333], 32)
    e = Decode(18, [5, 1300, 0], 32)
    w = max(d.bt.shape[1], e.bt.shape[1])
    bt = torch.full((3, w), -1, dtype=torch.int32, device="cuda")
    q, lens = bf(d.q), i32(d.lens)
    bt[:, :d.bt.shape[1]] = i32(d.bt)
    n = max(d.N, e.N)
    cache = torch.full((n, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache[:d.N] = d.cache
    dsa.dsa_paged_decode(q, cache, bt, lens, 16, d.scale)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = dsa.dsa_paged_decode(q, cache, bt, lens, 16, d.scale)
    g.replay()
    d.check((out, lse))
    cache[:] = float("nan")
    cache[:e.N] = e.cache
    bt.fill_(-1)
    bt[:, :e.bt.shape[1]] = i32(e.bt)
    q.copy_(bf(e.q))
    lens.copy_(i32(e.lens))
    g.replay()
    e.check((out, lse))


def test_decode_refusals():
    import dsa_sparse_mla_prefill_gb300 as dsa
    d = Decode(19, [50, 60], 16)
    q, bt, lens = bf(d.q), i32(d.bt), i32(d.lens)

    def call(**kw):
        a = dict(dict(q=q, cache=d.cache, bt=bt, lens=lens, idx=None, kw={}), **kw)
        return dsa.dsa_paged_decode(a["q"], a["cache"], a["bt"], a["lens"], 16, 1.0, idx=a["idx"], **a["kw"])
    for bad in (dict(q=q.transpose(0, 1)), dict(lens=lens[:1]), dict(bt=bt[:1]), dict(cache=d.cache[:, ::2]),
                dict(cache=torch.zeros(4, 600, dtype=torch.uint8, device="cuda")), dict(idx=i32(np.zeros((1, 4)))),
                dict(kw=dict(k=4)), dict(kw=dict(out=torch.zeros(2, 16, 256, dtype=torch.bfloat16, device="cuda"))),
                dict(lens=lens.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(lens=lens.long())
    for bad in (dict(q=torch.zeros(2, 129, 576, dtype=torch.bfloat16, device="cuda")),
                dict(q=torch.zeros(2, 16, 320, dtype=torch.bfloat16, device="cuda")),
                dict(idx=i32(np.zeros((2, 4))), kw=dict(k=5)),
                dict(kw=dict(workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(dsa.DSAError):
            call(**bad)


def test_decode_no_listed_positions():
    """k = 0 and an idx without columns: no keys, whatever the lengths."""
    d = Decode(22, [50, 3], 16)
    for idx in (torch.zeros(2, 0, dtype=torch.int32, device="cuda"), torch.zeros(2, 5, dtype=torch.int32, device="cuda")):
        out, lse = d.run(idx=idx, k=0)
        assert bad_count() == 0 and (out == 0).all() and torch.isneginf(lse).all()


def test_decode_position_listed_twice_counts_twice():
    d = Decode(23, [40], 16, k=6)
    d.idx[0, :6] = [7, 7, 3, -1, 7, 39]
    d.check(d.run())


def test_decode_shared_pages_and_many_requests():
    """Requests with a common prefix in the same pages; thousands of short requests."""
    d = Decode(24, [300] * 40, 32)
    d.bt[:, :10] = d.bt[0, :10]
    d.check(d.run())
    rng = np.random.default_rng(25)
    e = Decode(26, [160], 16)
    lens = rng.integers(0, 3, 5000).astype(np.int32) * 30 + rng.integers(0, 2, 5000).astype(np.int32)
    e.lens, e.bt = lens, np.repeat(e.bt, 5000, axis=0)
    e.q = normal_bf16(rng, (5000, 16, 576))
    e.check(e.run())


@pytest.mark.parametrize("gap", [31, 32, 33, 700])
def test_decode_long_runs_of_empty_requests(gap):
    """A padded batch: few requests have keys, the ones between them none."""
    rng = np.random.default_rng(28 + gap)
    d = Decode(28, [300], 16)
    B = 5 * gap + 7
    d.lens = np.where(np.arange(B) % gap == gap - 1, 290, 0).astype(np.int32)
    d.bt = np.repeat(d.bt, B, axis=0)
    d.q = normal_bf16(rng, (B, 16, 576))
    d.check(d.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_offsets_past_32_bits(fmt):
    """A cache of more than 4 GB whose pages lie at its ends: row offsets in bytes pass 2^32."""
    d = Decode(27, [700, 90], 32, bs=64, fmt=fmt)
    width = d.cache.shape[1] * d.cache.element_size()
    N = (2 ** 32 // width // 64 + 40) * 64
    big = torch.empty(N, d.cache.shape[1], dtype=d.cache.dtype, device="cuda")
    pages = int(d.N) // 64
    last = N // 64 - pages
    big[last * 64:] = d.cache
    assert last * 64 * width > 2 ** 32
    values = d.values
    d.cache = big
    bt = d.bt.copy()
    d.bt = np.where(bt >= 0, bt + last, -1).astype(np.int32)
    got = d.run()
    d.bt, d.N = bt, pages * 64
    d.values = values
    d.check(got)


def test_rope_and_append_offsets_past_32_bits():
    import dsa_sparse_mla_prefill_gb300 as dsa
    fr = dsa.dsa_rope_freqs(64)
    big = torch.empty(9, 2 ** 28 + 64, dtype=torch.bfloat16, device="cuda")           # 4.8 GB
    x = big[:, :128].unflatten(1, (2, 64))
    x.normal_()
    keep = x.clone()
    pos = np.arange(9, dtype=np.int32) * 1000
    dsa.dsa_rope(x, i32(pos), fr, out=x)
    check_rope(x, keep, pos, O.rope_frequencies(64, 10000.0), "interleaved")
    N = 2 ** 32 // 1152 + 100
    cache = big.flatten()[:N * 576].view(N, 576)
    rng = np.random.default_rng(3)
    c, pe = normal_bf16(rng, (2, 512)), normal_bf16(rng, (2, 64))
    bt = np.array([[N - 1, 0]], dtype=np.int32)
    dsa.dsa_kv_append(bf(c), bf(pe), i32([0, 1]), i32(bt), 1, cache, token_req=i32([0, 0]))
    assert bad_count() == 0
    assert np.array_equal(bits(cache[N - 1:]), np.concatenate([c[:1], pe[:1]], 1))
    assert np.array_equal(bits(cache[:1]), np.concatenate([c[1:], pe[1:]], 1))


def test_append_fp8_of_odd_values_is_the_quantize_kernels():
    """NaN, infinities, subnormals, zeros: the same bits as quantizing the bf16 row."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(8)
    c = rng.integers(0, 2 ** 16, (64, 512)).astype(np.uint16)          # any bf16 pattern
    c[0, :128], c[0, 128:256], c[0, 256:384] = 0x7fc0, 0x7f80, 0x8000   # a block of NaN, of infinities, of -0
    c[1, :128] = np.arange(128)                                          # subnormals
    c[2, :128], c[2, 5] = 0x7fc0, 0x3f80                                 # one number among NaN
    pe = normal_bf16(rng, (64, 64))
    f8 = torch.zeros(64, 656, dtype=torch.uint8, device="cuda")
    bt = i32(np.arange(64)[None])
    dsa.dsa_kv_append(bf(c), bf(pe), i32(np.arange(64)), bt, 1, f8, token_req=i32(np.zeros(64)))
    want = dsa.dsa_kv_fp8_quantize(bf(np.concatenate([c, pe], 1)), 64)
    assert bad_count() == 0 and torch.equal(f8, want)


def test_decode_two_graphs_at_once():
    """Two captured calls with their own workspaces, replayed on two streams together, and an eager call
    beside them."""
    ds = [Decode(30, [2500, 70, 900], 32), Decode(31, [4000], 16), Decode(32, [10, 1300], 64)]
    graphs, outs = [], []
    for d in ds[:2]:
        q, cache, bt, lens = bf(d.q), d.cache, i32(d.bt), i32(d.lens)
        import dsa_sparse_mla_prefill_gb300 as dsa
        dsa.dsa_paged_decode(q, cache, bt, lens, 16, d.scale)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dsa.dsa_paged_decode(q, cache, bt, lens, 16, d.scale))
        graphs.append((g, q, bt, lens))
    s = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    eager = None
    for _ in range(5):
        for (g, *_), st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(s[2]):
            eager = ds[2].run()
    torch.cuda.synchronize()
    for d, o in zip(ds, outs + [eager]):
        d.check(o)


def test_decode_head_pairs_in_graphs_at_once():
    """CTA pairs in two captured graphs on two streams, and a call over FP8 rows beside them."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    ds = [Decode(33, [2500, 70, 900], 128), Decode(34, [4000], 70, bs=64), Decode(35, [10, 1300], 16, fmt="fp8")]
    held, s = [], [torch.cuda.Stream() for _ in range(3)]
    for d in ds[:2]:
        args = (bf(d.q), d.cache, i32(d.bt), i32(d.lens), d.bs, d.scale)
        dsa.dsa_paged_decode(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = dsa.dsa_paged_decode(*args)
        held.append((g, out, args))
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, *_), st in zip(held, s):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(s[2]):
            third = ds[2].run()
    torch.cuda.synchronize()
    for d, o in zip(ds, [held[0][1], held[1][1], third]):
        d.check(o)


# ---------------------------------------------------------------------------
# the step: rotate the queries, append the new rows, attend
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k", [0, 64])
def test_decode_step(fmt, k):
    """Three generated tokens of four requests (one joins late, one row of the batch is padding), each
    a captured graph's replay, against the oracle run on the same cache."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(20 + k)
    H, bs, B = 32, 16, 4
    lens = np.array([130, 15, 400, 0], dtype=np.int32)
    bt, N = table_of(rng, lens + 8, bs)
    d0 = Decode(21, [1], H, bs=bs)   # (the checks below)
    f, layout = O.rope_frequencies(64, 10000.0, "yarn", 4.0), "interleaved"
    fr = dsa.dsa_rope_freqs(64, layout=layout, scaling="yarn", factor=4.0)
    kv = normal_bf16(rng, (N, 576))
    cache = bf(kv) if fmt == "bf16" else torch.from_numpy(O.kv_fp8_quantize(kv, 64)).cuda()
    x = torch.zeros(B, 576, dtype=torch.bfloat16, device="cuda")            # the new tokens' c_kv | k_pe
    qp = torch.zeros(B, H, 192, dtype=torch.bfloat16, device="cuda")        # projected queries, last 64 rotary
    q = torch.zeros(B, H, 576, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    kvl, btd = torch.zeros_like(pos), i32(bt)
    idx = torch.full((B, max(k, 1)), -1, dtype=torch.int32, device="cuda")

    def step():
        dsa.dsa_rope(qp[..., 128:], pos, fr, out=q[..., 512:])
        dsa.dsa_kv_append(x[:, :512], x[:, 512:], pos, btd, bs, cache, rope=fr)
        return dsa.dsa_paged_decode(q, cache, btd, kvl, bs, 192 ** -0.5, idx=idx if k else None)
    pos.fill_(-1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step()
    for t in range(3):
        live = np.array([True, True, True, t >= 1])
        xb, qb, qn = normal_bf16(rng, (B, 576)), normal_bf16(rng, (B, H, 192)), normal_bf16(rng, (B, H, 512))
        p = np.where(live, lens, -1).astype(np.int32)
        lens = lens + live
        x.copy_(bf(xb)), qp.copy_(bf(qb)), pos.copy_(i32(p)), kvl.copy_(i32(lens))
        q[..., :512] = bf(qn)
        ib = np.full((B, max(k, 1)), -1, dtype=np.int32)
        for b in range(B):
            m = min(k, int(lens[b]))
            ib[b, :m] = rng.permutation(int(lens[b]))[:m]
        idx.copy_(i32(ib))
        before = cache.clone()
        g.replay()
        torch.cuda.synchronize()
        # the cache: only the new rows changed
        rows, bad = O.append_rows(p, None, bt, bs, N)
        assert bad == 0
        keep = np.setdiff1d(np.arange(N), rows[rows >= 0])
        assert torch.equal(cache[keep.tolist()], before[keep.tolist()])
        r = rows[live]
        if fmt == "bf16":
            host = bits(cache)
            assert np.array_equal(host[r, :512], xb[live, :512])
            check_rows(host[r, 512:], xb[live, 512:], p[live], f, layout, 1.0)
        else:
            host = cache.cpu().numpy()
            assert np.array_equal(host[r, :528], O.kv_fp8_quantize(xb[live, :512], 0))
            host = O.kv_fp8_dequantize(host, 64)
        # the queries, then the attention over what the cache holds
        qg = q.clone()
        check_rope(qg[live][..., 512:], bf(qb[live])[..., 128:], p[live], f, layout)
        d0.q, d0.values, d0.bt, d0.lens = bits(qg), O.bf16_to_f64(host), bt, lens
        d0.idx, d0.k, d0.scale, d0.bs = (ib if k else None), k, 192 ** -0.5, bs
        d0.check((out, lse))
