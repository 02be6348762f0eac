"""Norms in front of the rotation and the step that checks drafted tokens, on the
GPU against the 64-bit oracle; edges of each, streams, captured graphs, and the
operators run as one step.

Tolerances, from the arithmetic (u = 2^-24, half a step of float32; a bf16
rounding is off by at most 2^-8 of the value):
  norm      a row's sum of squares is at most 72 products and additions one
            after another (a lane's up to 64 columns, five exchanges), 144 u of
            it; 1/n, the product, eps and the 2-ulp reciprocal root bring r
            within 80 u of itself; r and the weight round twice more: 82 u |n_c|
            per normed value.  Turning adds 10 u of |m| (|a| + |b|) (see
            test_gpu_decode_step.py): 92 u |m| (|a| + |b|) per turned output,
            then the bf16 rounding.
  gradient  G_c = |g_c|, in turned columns |m| (|g_a| + |g_b|): g is within 10 u
            G of the exact.  The sum S = sum g w x has the chain of the sum of
            squares and three roundings a term: 157 u A, A = sum G |w x|.  r g w:
            (80 + 10 + 3) u r G |w|.  x r^3 S / n: r^3 within 243 u, so 405 u
            |x| r^3 A / n with its products.  Their difference: one more u of each.
            dw: terms within 95 u of G |x| r, N of them added in some order:
            (95 + N) u sum G |x| r.
  tree      as the decode step's attention (test_gpu_decode_step.py).
"""
import ctypes
import math

import numpy as np
import pytest

import oracle.dsa_oracle as O
from gpu_util import bf, f32, i32, need_gpu, torch
from synth import normal_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


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


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# norms with rotation, and their gradient
# ---------------------------------------------------------------------------
class Norm:
    def __init__(self, seed, T, Hq, Hk, d, d_norm=None, d_rope=64, layout="interleaved", dtype=BF, w_dtype=None, mscale=1.3,
                 eps=1e-5, scale=1.0):
        import dsa_sparse_mla_prefill_gb300 as dsa
        rng = np.random.default_rng(seed)
        self.T, self.d, self.d_norm, self.d_rope, self.layout, self.eps, self.dtype = T, d, d_norm or d, d_rope, layout, eps, dtype
        self.given = d_norm

        def make(*shape, by=1.0):
            return torch.from_numpy((rng.standard_normal(shape) * by).astype(np.float32)).cuda().to(dtype)
        self.x = [make(T, H, d, by=scale) if H else None for H in (Hq, Hk)]
        self.g = [make(T, H, d) if H else None for H in (Hq, Hk)]
        self.w = [(make(self.d_norm) + 1).to(w_dtype or dtype) if H else None for H in (Hq, Hk)]
        self.pos = rng.integers(-1000, 200000, T).astype(np.int32)
        self.f = O.rope_frequencies(d_rope, 10000.0) if d_rope else None
        self.m = float(np.float32(mscale)) if d_rope else 1.0
        self.freqs = dsa.dsa_rope_freqs(d_rope, layout=layout, mscale=mscale) if d_rope else None

    def forward(self, **kw):
        import dsa_sparse_mla_prefill_gb300 as dsa
        return dsa.dsa_qk_norm_rope(*self.x, *self.w, i32(self.pos) if self.d_rope else None, self.freqs, eps=self.eps,
                                    d_norm=self.given, **kw)

    def gradient(self, **kw):
        import dsa_sparse_mla_prefill_gb300 as dsa
        return dsa.dsa_qk_norm_rope_gradient(*self.g, *self.x, *self.w, i32(self.pos) if self.d_rope else None, self.freqs,
                                             eps=self.eps, d_norm=self.given, **kw)

    def paired(self, v):
        """|v|, in turned columns |m| (|a| + |b|)."""
        v = np.abs(v)
        if self.d_rope:
            r = self.d - self.d_rope
            a = v[..., r:]
            if self.layout == "interleaved":
                p = np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)
            else:
                p = np.tile(a[..., :self.d_rope // 2] + a[..., self.d_rope // 2:], 2)
            v = np.concatenate([v[..., :r], self.m * p], -1)
        return v

    def within(self, got, want, tol):
        if got.dtype is BF:
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        err = np.abs(f64(got) - want)
        assert (err <= tol + 1e-37).all(), float((err - tol).max())

    def check_forward(self, got):
        for x, w, y in zip(self.x, self.w, got):
            if x is None:
                assert y is None
                continue
            args = (f64(x), f64(w), self.pos, self.f, self.layout, self.eps, self.d_norm)
            want = O.norm_rope(*args, self.m)
            unturned = O.norm_rope(*args[:3], None, *args[4:])
            self.within(y, want, 92 * U * self.paired(unturned))

    def check_gradient(self, got):
        n = self.d_norm
        for x, w, g, gx, gw in zip(self.x, self.w, self.g, got[:2], got[2:]):
            if x is None:
                assert gx is None and gw is None
                continue
            xd, wd, gd = f64(x), f64(w), f64(g)
            want, want_w = O.norm_rope_gradient(gd, xd, wd, self.pos, self.f, self.layout, self.eps, n, self.m)
            G = self.paired(gd)
            r = 1 / np.sqrt((xd[..., :n] ** 2).mean(-1, keepdims=True) + self.eps)
            A = (G[..., :n] * np.abs(wd * xd[..., :n])).sum(-1, keepdims=True)
            tol = 10 * U * G
            tol[..., :n] = 94 * U * r * G[..., :n] * np.abs(wd) + 406 * U * np.abs(xd[..., :n]) * r ** 3 * A / n
            self.within(gx, want, tol)
            terms = (G[..., :n] * np.abs(xd[..., :n]) * r).sum(axis=(0, 1))
            self.within(gw, want_w, (95 + x.shape[0] * x.shape[1]) * U * terms)


NORM_CASES = [
    # T, Hq, Hk, d, d_norm, d_rope: whole heads, latent rows, no turning, all turned, norm ends inside the turned columns
    (1, 16, 1, 192, None, 64), (7, 1, 0, 576, 512, 64), (33, 4, 4, 256, None, 0), (5, 3, 2, 128, None, 128),
    (9, 0, 5, 192, 160, 64), (300, 2, 1, 64, 64, 64), (2, 1, 1, 1024, None, 256), (3, 2, 2, 512, 8, 32), (17, 8, 1, 256, None, 256),
    # columns that no 16-byte piece divides
    (4, 3, 2, 70, None, 6), (3, 1, 2, 1, None, 0), (6, 2, 0, 37, 5, 36), (2, 1, 1, 1023, 1022, 254), (5, 2, 2, 72, None, 8)]


@pytest.mark.parametrize("case", NORM_CASES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_and_gradient(case, layout, dtype):
    T, Hq, Hk, d, d_norm, d_rope = case
    c = Norm(d + T, T, Hq, Hk, d, d_norm, d_rope, layout, dtype)
    keep = [None if x is None else x.clone() for x in c.x]
    c.check_forward(c.forward())
    c.check_gradient(c.gradient())
    assert all(x is None or torch.equal(x, y) for x, y in zip(c.x, keep))


@pytest.mark.parametrize("T,Hq,Hk", [(2500, 5, 3), (1, 300, 2), (4001, 1, 0), (70, 64, 8)])
@pytest.mark.parametrize("dtype,w_dtype", [(BF, F32), (F32, BF)])
def test_norm_many_rows(T, Hq, Hk, dtype, w_dtype):
    """Rows that are dealt unevenly, weights of the other type."""
    c = Norm(T, T, Hq, Hk, 128, None, 64, "half", dtype, w_dtype)
    c.check_forward(c.forward())
    c.check_gradient(c.gradient())


def test_norm_sizes_of_x():
    """Rows of zeros, tiny and large values, eps of zero."""
    for scale, eps in ((0.0, 1e-6), (1e-12, 1e-6), (1e15, 1e-6), (3.0, 0.0), (1e-3, 100.0)):
        c = Norm(3, 6, 2, 1, 192, dtype=F32, eps=eps, scale=scale)
        c.check_forward(c.forward())
        if scale >= 1e-3:
            c.check_gradient(c.gradient())


@pytest.mark.parametrize("d,T", [(64, 7), (128, 1), (256, 33), (576, 3)])
def test_norm_gradient_without_eps_where_lanes_lack_rows(d, T):
    """eps = 0 with fewer rows than the groups of lanes take at a time: those without one add nothing."""
    for dtype in (BF, F32):
        c = Norm(d + T, T, 1, 3, d, None, 0, dtype=dtype, eps=0.0)
        c.check_forward(c.forward())
        c.check_gradient(c.gradient())


def test_norm_views_and_places():
    """Columns of a wider projection, in place, odd offsets, broadcast inputs, results in the caller's tensors."""
    c = Norm(8, 20, 3, 2, 192)
    q, k = c.x
    both = torch.randn(20, 5, 400, device="cuda", dtype=BF)
    both[:, :3, 200:392], both[:, 3:, 200:392] = q, k
    around = both.clone()
    c.x = [both[:, :3, 200:392], both[:, 3:, 200:392]]
    want = c.forward()
    c.check_forward(want)
    c.check_gradient(c.gradient())
    got = c.forward(q_out=c.x[0], k_out=c.x[1])
    assert got[0] is c.x[0] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    around[:, :, 200:392] = torch.cat(want, 1)
    assert torch.equal(both, around)                                    # nothing beside the columns
    # rows that no 16-byte access fits: other results only by the order of the sums
    odd = torch.zeros(20, 3, 193, device="cuda", dtype=BF)
    odd[..., 1:] = q
    c.x = [odd[..., 1:], k]
    c.check_forward(c.forward())
    c.check_gradient(c.gradient())
    # one row for every head, gradients that are one number
    c.x = [q[:, :1].expand(20, 3, 192), k[:1].expand(20, 2, 192)]
    c.g = [c.g[0][:1, :1].expand(20, 3, 192), c.g[1]]
    c.check_forward(c.forward())
    c.check_gradient(c.gradient())


def test_norm_gradient_is_the_difference_quotient():
    c = Norm(9, 4, 2, 1, 128, None, 64, "half", F32)
    got = c.gradient()

    def loss(x, w):
        c2 = [O.norm_rope(f64(a), f64(b), c.pos, c.f, c.layout, c.eps, c.d_norm, c.m) for a, b in zip(x, w)]
        return sum((f64(g) * y).sum() for g, y in zip(c.g, c2))
    rng = np.random.default_rng(1)
    for which, grads in ((0, got[:2]), (1, got[2:])):
        step = [torch.from_numpy(rng.standard_normal(tuple(t.shape))).cuda() for t in (c.x, c.w)[which]]
        h = 1e-4
        up = [t.double() + h * s for t, s in zip((c.x, c.w)[which], step)]
        down = [t.double() - h * s for t, s in zip((c.x, c.w)[which], step)]
        a = loss(up, c.w) if which == 0 else loss(c.x, up)
        b = loss(down, c.w) if which == 0 else loss(c.x, down)
        want = sum((f64(g) * f64(s)).sum() for g, s in zip(grads, step))
        size = sum((np.abs(f64(g)) * np.abs(f64(s))).sum() for g, s in zip(grads, step))
        # the third derivatives along the step are below 100 of the gradient's size: h^2 100 / 6 of it, and rounding
        assert abs((a - b) / (2 * h) - want) <= (h * h * 20 + 600 * U) * size


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_gradient_gives_the_same_bits(dtype):
    c = Norm(10, 1500, 4, 2, 192, dtype=dtype)
    import dsa_sparse_mla_prefill_gb300 as dsa
    ws = torch.full((dsa.dsa_qk_norm_rope_gradient_workspace(192),), 255, dtype=torch.uint8, device="cuda")
    a = c.gradient()
    for _ in range(3):
        b = c.gradient(workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_norm_nothing_to_do_and_refusals():
    import dsa_sparse_mla_prefill_gb300 as dsa
    c = Norm(11, 0, 3, 2, 192)
    out = c.forward()
    assert out[0].shape == (0, 3, 192) and out[1].shape == (0, 2, 192)
    gq, gk, gqw, gkw = c.gradient()
    assert gq.shape == (0, 3, 192) and (gqw == 0).all() and (gkw == 0).all()
    c = Norm(12, 5, 3, 2, 192)
    q, k = c.x
    c.x = [q[:, :0], k]                                                 # no heads on one side
    c.g = [c.g[0][:, :0], c.g[1]]
    assert c.forward()[0].shape == (5, 0, 192)
    gq, gk, gqw, gkw = c.gradient()
    assert gq.shape == (5, 0, 192) and (gqw == 0).all() and (gkw != 0).any()
    w, pos, fr = c.w[0], i32(c.pos), c.freqs

    def call(**kw):
        a = dict(dict(q=q, k=k, qw=w, kw=w, pos=pos, fr=fr, more={}), **kw)
        return dsa.dsa_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["fr"], **a["more"])
    call()
    for bad in (dict(k=k[:3]), dict(k=k[..., :128]), dict(k=k.float()), dict(kw=w.float()), dict(qw=w[:100]), dict(pos=pos[:2]),
                dict(q=q[..., ::2], k=None), dict(more=dict(d_norm=193)), dict(more=dict(d_norm=0)), dict(more=dict(q_out=k)),
                dict(k=None, more=dict(k_out=k)), dict(fr=dsa.dsa_rope_freqs(194)), dict(pos=pos.cpu()), dict(qw=w.cpu()),
                dict(q=q[0])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(qw=None), dict(q=q.half()), dict(fr=3), dict(pos=None)):
        with pytest.raises(TypeError):
            call(**bad)
    both = torch.empty_like(k)
    for bad in (dict(more=dict(eps=-1.0)), dict(more=dict(eps=math.nan)), dict(more=dict(eps=math.inf)),
                dict(more=dict(q_out=q[:, :1].expand(5, 3, 192))), dict(q=k, more=dict(q_out=both, k_out=both))):
        with pytest.raises(dsa.DSAError):
            call(**bad)
    big = torch.zeros(1, 1, 1025, device="cuda")
    with pytest.raises(dsa.DSAError):
        dsa.dsa_qk_norm_rope(big, None, big[0, 0], None, None)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_qk_norm_rope_gradient(q, k, q, k, w, w, pos, fr, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))


def test_norm_offsets_past_32_bits():
    big = torch.empty(5, 2 ** 29 + 64, dtype=BF, device="cuda")            # 5.4 GB
    c = Norm(13, 5, 1, 0, 192)
    x = big[:, None, :192]
    x.copy_(c.x[0])
    c.x = [x, None]
    c.check_forward(c.forward())
    c.check_gradient(c.gradient())
    got = c.forward(q_out=big[:, None, 4096:4288])
    c.check_forward(got)


# ---------------------------------------------------------------------------
# tree
# ---------------------------------------------------------------------------
def ancestors(parent):
    """Mask words of a tree by each token's parent (-1: the context)."""
    m = []
    for j, p in enumerate(parent):
        m.append((m[p] if p >= 0 else 0) | 1 << j)
    return m


def signed(words):
    return np.array(words, dtype=np.uint64).view(np.int64)


def table_of(rng, lens, bs, spare=3):
    nb = [-(-int(n) // bs) for n in lens]
    ids = rng.permutation(sum(nb) + spare)
    bt = np.full((len(lens), max(max(nb), 1)), -1, dtype=np.int32)
    p = 0
    for r, n in enumerate(nb):
        bt[r, :n] = ids[p:p + n]
        p += n
    return bt, (sum(nb) + spare) * bs


class Tree:
    """Random trees over a shuffled paged cache whose rows that no token sees are NaN."""

    def __init__(self, seed, lens, n, H, bs=16, d_rope=64, fmt="bf16", scale=192 ** -0.5, spread=1.0, ld_extra=0, drafted=None,
                 mask=None):
        rng = np.random.default_rng(seed)
        self.lens, self.n, self.H, self.bs, self.scale = np.asarray(lens, dtype=np.int32), n, H, bs, scale
        B, d = len(lens), 512 + d_rope
        self.bt, self.N = table_of(rng, np.maximum(self.lens, 0), bs)
        self.drafted = None if drafted is None else np.asarray(drafted, dtype=np.int32)
        if mask is None:
            mask = [ancestors([int(rng.integers(-1, j)) if j else -1 for j in range(n)]) for _ in range(B)]
        self.mask = signed(mask)
        self.q = normal_bf16(rng, (B, n, H, d))
        if spread != 1.0:
            self.q = O._f32_to_bf16_bits((O.bf16_to_f64(self.q) * spread).astype(np.float32))
        kv = normal_bf16(rng, (self.N, d))
        used = np.zeros(self.N, dtype=bool)
        for b, length in enumerate(self.lens):
            nb = n if drafted is None else int(np.clip(self.drafted[b], 0, n))
            context = int(length) - nb
            words = [int(w) & (1 << 64) - 1 for w in self.mask[b][:nb]]
            for p in range(max(int(length), 0)):
                if p < context or any(w >> (p - context) & 1 for w in words):
                    used[self.bt[b, p // bs] * bs + p % bs] = True
        if fmt == "bf16":
            kv[~used] = 0x7fc0
            self.cache = torch.full((self.N, d + ld_extra), float("nan"), dtype=BF, device="cuda")
            self.cache[:, :d] = bf(kv)
            self.values = O.bf16_to_f64(kv)
        else:
            rows = O.kv_fp8_quantize(kv, d_rope)
            self.values = O.bf16_to_f64(O.kv_fp8_dequantize(rows, d_rope))
            rows[~used] = 0x7f
            self.cache = torch.from_numpy(rows).cuda()
        self.values[~used] = np.nan

    def args(self):
        return bf(self.q), self.cache, i32(self.bt), i32(self.lens), torch.from_numpy(self.mask).cuda(), self.bs, self.scale

    def run(self, **kw):
        import dsa_sparse_mla_prefill_gb300 as dsa
        if self.drafted is not None:
            kw = dict(dict(num_draft=i32(self.drafted)), **kw)
        return dsa.dsa_tree_decode(*self.args(), **kw)

    def check(self, got, bad=0):
        out, lse = got
        ref = O.tree_decode(self.q, self.values, self.bt, self.lens, self.mask, self.bs, self.scale, self.drafted)
        assert bad_count() == ref["bad"] == bad
        score = 1155 * U * ref["mass"]
        tol = (2 * (2.0 ** -8 + score) * (1 + 2.0 ** -7))[..., None] * ref["spread"] + 2.0 ** -8 * np.abs(ref["out"]) + 1e-30
        err = np.abs(f32(out) - ref["out"])
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
        assert (f32(out)[np.isinf(ref["lse"])] == 0).all()
        got_l, inf = f64(lse), np.isinf(ref["lse"])
        assert np.array_equal(inf, np.isneginf(got_l))
        tiles = -(-max(int(self.lens.max()), 1) // 128)
        ltol = score + 2.0 ** -21 + (tiles + 32) * U + 4 * U * np.where(inf, 0, np.abs(ref["lse"]))
        lerr = np.abs(np.where(inf, 0, got_l) - np.where(inf, 0, ref["lse"]))
        assert (lerr <= ltol).all(), float((lerr / ltol).max())


FMTS = ["bf16", "fp8"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(1, 16), (3, 5), (2, 16), (11, 3), (4, 16), (5, 13), (8, 16), (5, 24), (2, 128), (64, 4), (16, 16)])
@pytest.mark.parametrize("lens", [[300], [128], [129, 0, 131], [70, 255, 64, 66]])
def test_tree_small(fmt, n, H, lens):
    t = Tree(n, lens, n, H, fmt=fmt)
    t.check(t.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H,d_rope,bs", [(7, 8, 64, 1), (8, 16, 0, 7), (3, 32, 64, 24), (4, 128, 64, 64), (16, 24, 0, 64),
                                           (33, 16, 64, 128), (12, 64, 64, 100), (64, 32, 64, 64), (16, 128, 0, 16), (2, 65, 64, 256)])
def test_tree_shapes(fmt, n, H, d_rope, bs):
    """Rows that fill no block of them, all page sizes, wider cache rows, lengths at tile borders."""
    t = Tree(H, [700, 64, 0, 257, 1024 + n // 2, 128 + n], n, H, bs=bs, d_rope=d_rope, fmt=fmt, ld_extra=8)
    t.check(t.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(2, 8), (4, 8), (4, 16), (8, 16), (8, 32), (4, 128)])
def test_tree_long_context_is_split(fmt, n, H):
    t = Tree(7, [20011], n, H, bs=64, fmt=fmt)
    t.check(t.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(4, 8), (6, 16), (8, 24), (40, 16)])
def test_tree_ragged(fmt, n, H):
    """Requests with fewer drafted tokens, none, more than positions; padding requests."""
    rng = np.random.default_rng(n)
    lens = np.array([500, 3, 0, 2 * n, 129, 1, -4, 260, 128, 2000], dtype=np.int32)
    drafted = np.array([1, n, n, 0, n // 2, 2, 3, n + 5, -1, n], dtype=np.int32)
    t = Tree(n, lens, n, H, fmt=fmt, drafted=drafted, bs=int(rng.integers(1, 70)))
    t.check(t.run())


@pytest.mark.parametrize("n,H", [(5, 3), (5, 6), (5, 9), (5, 16), (9, 16), (3, 64)])
def test_tree_masks(n, H):
    """Tokens that see nothing, not themselves, later ones; bits behind the last token; no context at all."""
    words = [[0, 1, (1 << 64) - 1] + [1 << (n - 1)] * (n - 3), [0] * n, ancestors(range(-1, n - 1)), [(1 << 64) - 2] * n]
    for lens in ([200, 130, 128 + n // 2, 300], [n, n, n, n]):
        t = Tree(n, lens, n, H, mask=words)
        t.check(t.run())


@pytest.mark.parametrize("n,H", [(4, 8), (4, 16), (8, 32)])
def test_tree_wide_and_rising_scores(n, H):
    t = Tree(10, [900, 4000], n, H, spread=30.0)
    t.check(t.run())
    # the drafted tokens' own scores are the largest by far, and only some see them
    t = Tree(11, [1300, 260], n, H)
    for b, length in enumerate(t.lens):
        for j in range(n):
            p = int(length) - n + j
            r = int(t.bt[b, p // 16] * 16 + p % 16)
            v = O._f32_to_bf16_bits((O.bf16_to_f64(t.q)[b, (j + 1) % n, 0] * 6).astype(np.float32))
            t.values[r] = O.bf16_to_f64(v)
            t.cache[r, :576] = bf(v)
    t.check(t.run())
    for scale in (-0.05, 0.0):
        t = Tree(12, [300, 1300], n, H, scale=scale)
        t.check(t.run())


@pytest.mark.parametrize("fmt", FMTS)
def test_tree_bad_entries_are_absent(fmt):
    t = Tree(13, [200, 90, 64, 500], 8, 16, fmt=fmt)
    t.bt[3, 2], t.bt[3, 5] = -4, t.N // 16
    t.bt[1, 5] = -1                                                    # the page of the drafted tokens
    seen = t.mask[1].astype(np.uint64)
    gone = sum(1 for p in range(80, 90) if p < 82 or any(int(w) >> (p - 82) & 1 for w in seen))
    t.check(t.run(), bad=32 + gone)
    # a length past the table is cut, the drafted tokens behind it with it
    t.lens[2] = 10 ** 6
    t.check(t.run(), bad=32 + gone + 1 + (t.bt.shape[1] - 4) * 16)
    t.bt[:] = -1
    t.lens[:] = [8, 0, -5, 9]
    t.check(t.run(), bad=17)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(2, 16), (3, 16), (5, 16), (9, 16)])
def test_tree_queries_of_other_rows_stay_there(fmt, n, H):
    """NaN and infinite queries of padding requests and of one token's first head reach no other row."""
    t = Tree(21, [300, 0, 700, 0], n, H, fmt=fmt)
    want = t.run()
    t.check(want)
    t.q[1], t.q[3] = 0x7fc0, 0x7f80
    t.q[2, n - 1, 0] = 0x7fc0
    out, lse = t.run()
    keep = torch.ones(4, n, H, dtype=torch.bool, device="cuda")
    keep[2, n - 1, 0] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])
    assert torch.isnan(out[~keep]).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [4, 16, 64])
def test_tree_empty(fmt, H):
    import dsa_sparse_mla_prefill_gb300 as dsa
    q = bf(normal_bf16(np.random.default_rng(1), (2, 3, H, 576)))
    cache = torch.empty(0, 576, dtype=BF, device="cuda") if fmt == "bf16" else torch.empty(0, 656, dtype=torch.uint8, device="cuda")
    mask = torch.tensor([[1, 2, 4], [1, 3, 7]], device="cuda")
    for bs in (16, 3):
        out, lse = dsa.dsa_tree_decode(q, cache, i32([[0, 0], [0, 0]]), i32([5, 0]), mask, bs, 1.0)
        assert bad_count() == 5 and (out == 0).all() and torch.isneginf(lse).all()
    out, lse = dsa.dsa_tree_decode(q[:0], cache, i32(np.zeros((0, 1))), i32(np.zeros(0)), mask[:0], 16, 1.0)
    assert out.shape == (0, 3, H, 512)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(4, 8), (4, 16), (8, 16), (4, 128)])
def test_tree_same_bits_and_shared_workspace(fmt, n, H):
    import dsa_sparse_mla_prefill_gb300 as dsa
    t, e = Tree(14, [3000, 777, 129], n, H, fmt=fmt), Tree(15, [2500], n, H, fmt=fmt)
    ws = torch.full((dsa.dsa_tree_decode_workspace(3, n, H, t.bt.shape[1] * 16),), 255, dtype=torch.uint8, device="cuda")
    a = t.run(workspace=ws)
    e.check(e.run(workspace=ws))
    b = t.run(workspace=ws)
    for _ in range(10):
        c = t.run(workspace=ws)
    torch.cuda.synchronize()
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    t.check(b)


def test_tree_of_one_token_is_decode():
    import dsa_sparse_mla_prefill_gb300 as dsa
    t = Tree(16, [500, 33, 0, 2000], 1, 32)
    out, lse = t.run()
    q, cache, bt, lens, _, bs, scale = t.args()
    want = dsa.dsa_paged_decode(q[:, 0], cache, bt, lens, bs, scale)
    assert torch.equal(out[:, 0], want[0]) and torch.equal(lse[:, 0], want[1])


@pytest.mark.parametrize("n,H", [(4, 8), (4, 16), (8, 16), (2, 128)])
def test_tree_on_another_stream_and_outputs_kept(n, H):
    t = Tree(17, [500, 1500], n, H)
    big, lse = torch.full((4, n, H, 512), 5.0, dtype=BF, device="cuda"), torch.full((4, n, H), 5.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = t.run(out=big[:2], lse=lse[:2], stream=s)
    s.synchronize()
    t.check(got)
    assert (big[2:] == 5).all() and (lse[2:] == 5).all()
    with torch.cuda.stream(s):
        got = t.run()
    s.synchronize()
    t.check(got)


@pytest.mark.parametrize("n,H", [(4, 8), (4, 16), (8, 16)])
def test_tree_graph_follows_its_tensors(n, H):
    """One captured call, replayed as lengths, tables, masks and numbers of drafted tokens change."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    a, b = Tree(18, [900, 40, 333], n, H, drafted=[n, 2, 1]), Tree(19, [9, 1300, 0], n, H, drafted=[n, n - 1, n])
    w, N = max(a.bt.shape[1], b.bt.shape[1]), max(a.N, b.N)
    held = [t.clone() for t in (bf(a.q), i32(a.lens), torch.from_numpy(a.mask).cuda(), i32(a.drafted))]
    bt = torch.full((3, w), -1, dtype=torch.int32, device="cuda")
    cache = torch.full((N, 576), float("nan"), dtype=BF, device="cuda")

    def step():
        return dsa.dsa_tree_decode(held[0], cache, bt, held[1], held[2], 16, a.scale, num_draft=held[3])
    held[1].fill_(0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in (a, b, a):
        for dst, src in zip(held, (bf(t.q), i32(t.lens), torch.from_numpy(t.mask).cuda(), i32(t.drafted))):
            dst.copy_(src)
        bt.fill_(-1)
        bt[:, :t.bt.shape[1]] = i32(t.bt)
        cache.fill_(float("nan"))
        cache[:t.N] = t.cache
        g.replay()
        t.check(got)


def test_tree_graphs_at_once():
    """Two captured calls with their own workspaces on two streams, an eager call beside them."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    ts = [Tree(30, [2500, 70, 900], 8, 16), Tree(31, [4000], 4, 128, bs=64), Tree(32, [70, 1300], 5, 16, fmt="fp8")]
    held, s = [], [torch.cuda.Stream() for _ in range(3)]
    for t in ts[:2]:
        args = t.args()
        dsa.dsa_tree_decode(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = dsa.dsa_tree_decode(*args)
        held.append((g, out, args))
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, *_), st in zip(held, s):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(s[2]):
            third = ts[2].run()
    torch.cuda.synchronize()
    for t, o in zip(ts, [held[0][1], held[1][1], third]):
        t.check(o)


def test_calls_from_two_threads():
    """Two host threads with a stream each, calling the operators at the same time."""
    import threading
    ts = [Tree(40, [900, 33, 2000], 4, 16), Tree(41, [1500, 260], 9, 16, fmt="fp8", bs=64)]
    ns = [Norm(42, 300, 4, 2, 192), Norm(43, 77, 8, 1, 128, None, 64, "half", F32)]
    want = [(*t.run(), *c.forward(), *c.gradient()) for t, c in zip(ts, ns)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = (*ts[i].run(), *ns[i].forward(), *ns[i].gradient())
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong
    for t, w in zip(ts, want):
        t.check(w[:2])


@pytest.mark.parametrize("most", [300, 1500])
@pytest.mark.parametrize("n,H", [(4, 8), (3, 16), (8, 16)])
def test_tree_many_requests(n, H, most):
    """Hundreds of short requests, padding ones in long runs among them."""
    rng = np.random.default_rng(5)
    lens = np.where(rng.random(400) < 0.3, rng.integers(n, most, 400), 0).astype(np.int32)
    t = Tree(20, lens, n, H)
    t.check(t.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,H", [(4, 8), (8, 16)])
def test_tree_offsets_past_32_bits(fmt, n, H):
    t = Tree(27, [700, 90], n, H, bs=64, fmt=fmt)
    width = t.cache.shape[1] * t.cache.element_size()
    N = (2 ** 32 // width // 64 + 40) * 64
    big = torch.empty(N, t.cache.shape[1], dtype=t.cache.dtype, device="cuda")
    pages = int(t.N) // 64
    last = N // 64 - pages
    big[last * 64:] = t.cache
    t.cache, bt = big, t.bt.copy()
    t.bt = np.where(bt >= 0, bt + last, -1).astype(np.int32)
    got = t.run()
    t.bt, t.N = bt, pages * 64
    t.check(got)


def test_tree_refusals():
    import dsa_sparse_mla_prefill_gb300 as dsa
    t = Tree(19, [50, 60], 4, 16)
    q, cache, bt, lens, mask, bs, scale = t.args()

    def call(**kw):
        a = dict(dict(q=q, cache=cache, bt=bt, lens=lens, mask=mask, kw={}), **kw)
        return dsa.dsa_tree_decode(a["q"], a["cache"], a["bt"], a["lens"], a["mask"], bs, scale, **a["kw"])
    for bad in (dict(q=q.transpose(1, 2)), dict(q=q[:, 0]), dict(lens=lens[:1]), dict(bt=bt[:1]), dict(mask=mask[:, :3]),
                dict(mask=mask.cpu()), dict(mask=mask.t().contiguous().t()), dict(cache=cache[:, ::2]),
                dict(kw=dict(num_draft=lens[:1])), dict(kw=dict(out=torch.zeros(2, 4, 16, 256, dtype=BF, device="cuda"))),
                dict(kw=dict(lse=torch.zeros(2, 4, 15, device="cuda"))), dict(lens=lens.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(lens=lens.long()), dict(mask=mask.int()), dict(kw=dict(num_draft=lens.long())), dict(q=q.float())):
        with pytest.raises(TypeError):
            call(**bad)
    zeros = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")
    for bad in (dict(q=zeros(2, 4, 129, 576)), dict(q=zeros(2, 65, 1, 576), mask=mask.repeat(1, 17)[:, :65].contiguous()),
                dict(q=zeros(2, 33, 64, 576), mask=mask.repeat(1, 9)[:, :33].contiguous()), dict(q=zeros(2, 4, 16, 320)),
                dict(kw=dict(workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(dsa.DSAError):
            call(**bad)


# ---------------------------------------------------------------------------
# keep
# ---------------------------------------------------------------------------
def random_path(rng, n, m):
    k = int(rng.integers(0, min(n, m) + 1))
    path = np.full(m, -1, dtype=np.int32)
    path[:k] = np.sort(rng.permutation(n)[:k])
    return path


@pytest.mark.parametrize("fmt,d_rope,extra", [("bf16", 64, 0), ("bf16", 0, 24), ("fp8", 64, 0), ("fp8", 0, 0)])
@pytest.mark.parametrize("layers,n,bs", [(1, 4, 16), (3, 64, 5), (61, 16, 64), (128, 7, 1)])
def test_keep(fmt, d_rope, extra, layers, n, bs):
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(layers + n)
    B, m = 9, min(n, 40)
    lens = (rng.integers(0, 50, B) + n).astype(np.int32)
    lens[4] = 0
    bt, N = table_of(rng, lens, bs)
    keep = np.stack([random_path(rng, n, m) for _ in range(B)])
    keep[0, :m] = np.arange(n - m, n)                                    # the last of all
    keep[1] = np.where(np.arange(m) < 2, np.arange(m) + min(1, n - 2), -1)  # each into the next one's place
    width = 512 + d_rope + extra if fmt == "bf16" else 528 + 2 * d_rope
    caches = [torch.from_numpy(rng.integers(0, 2 ** 16, (N, width)).astype(np.uint16).view(np.int16)).cuda().view(BF)
              if fmt == "bf16" else torch.from_numpy(rng.integers(0, 256, (N, width), dtype=np.uint8)).cuda() for _ in range(layers)]
    raw = torch.int16 if fmt == "bf16" else torch.uint8
    before = [c.view(raw).clone() for c in caches]
    got = dsa.dsa_kv_keep(caches if layers > 1 else caches[0], i32(bt), i32(lens), i32(keep), bs, n)
    moves, want, bad = O.kv_keep(bt, lens, keep, bs, N, n)
    assert bad_count() == bad == 0 and np.array_equal(got.cpu().numpy(), want)
    src, dst = [a for a, _ in moves], [b for _, b in moves]
    for c, old in zip(caches, before):
        new = old.clone()
        new[dst] = old[src]
        assert torch.equal(c.view(raw), new)


def test_keep_ragged_and_bad():
    """Numbers of drafted tokens, entries that are none, lost pages, padding requests, the caller's lengths."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(3)
    lens = np.array([20, 9, 0, -3, 4, 30, 30, 30, 30, 64, 30], dtype=np.int32)
    drafted = np.array([6, 3, 2, 2, 6, -1, 9, 8, 4, 8, 0], dtype=np.int32)
    bt, N = table_of(rng, np.maximum(lens, 1), 4)
    keep = np.array([[1, 3, 5, -1, 7], [0, 2, 3, -1, -1], [1, -1, -1, -1, -1], [0, 1, -1, -1, -1], [1, 2, -1, -1, -1],
                     [0, -1, -1, -1, -1], [-1, 0, 0, 0, 0], [3, 3, 4, 5, 6], [2, 1, -1, -1, -1], [1, 4, 5, 6, 7], [0, 1, 2, 3, 4]],
                    dtype=np.int32)
    bt[9, 14], bt[9, 15] = -1, N // 4 + 3
    cache = bf(normal_bf16(rng, (N, 576)))
    before = cache.clone()
    moves, want, bad = O.kv_keep(bt, lens, keep, 4, N, 8, drafted)
    new = torch.full((13,), 77, dtype=torch.int32, device="cuda")
    got = dsa.dsa_kv_keep(cache, i32(bt), i32(lens), i32(keep), 4, 8, num_draft=i32(drafted), new_lens=new[:11])
    assert bad_count() == bad and bad >= 6
    assert np.array_equal(got.cpu().numpy(), want) and (new[11:] == 77).all()
    ref = before.clone()
    ref[[b for _, b in moves]] = before[[a for a, _ in moves]]
    assert torch.equal(cache, ref)
    # nothing to do
    assert dsa.dsa_kv_keep(cache, i32(np.zeros((0, 1))), i32(np.zeros(0)), i32(np.zeros((0, 3))), 4, 8).shape == (0,)
    got = dsa.dsa_kv_keep(cache, i32(bt[:2]), i32(lens[:2]), i32(np.zeros((2, 0))), 4, 8)
    assert got.tolist() == [12, 1] and torch.equal(cache, ref)
    for wrong in (dict(keep=i32(keep[:3])), dict(caches=[cache, cache[:4]]), dict(caches=[cache, cache.float()]),
                  dict(caches=cache[:, ::2]), dict(new_lens=new)):
        a = dict(dict(caches=cache, keep=i32(keep), new_lens=None), **wrong)
        with pytest.raises(ValueError):
            dsa.dsa_kv_keep(a["caches"], i32(bt), i32(lens), a["keep"], 4, 8, new_lens=a["new_lens"])
    same = i32(lens)
    for wrong in (dict(caches=[cache, cache]), dict(n=65), dict(new_lens=same), dict(caches=[cache] * 129)):
        a = dict(dict(caches=cache, n=8, new_lens=None), **wrong)
        with pytest.raises(dsa.DSAError):
            dsa.dsa_kv_keep(a["caches"], i32(bt), same, i32(keep), 4, a["n"], new_lens=a["new_lens"])


def test_keep_offsets_past_32_bits():
    import dsa_sparse_mla_prefill_gb300 as dsa
    N = 2 ** 32 // 1152 + 100
    big = torch.empty(N, 576, dtype=BF, device="cuda")
    rows = bf(normal_bf16(np.random.default_rng(3), (4, 576)))
    big[N - 4:] = rows
    bt = np.array([[N - 4, N - 3, N - 2, N - 1]], dtype=np.int32)
    new = dsa.dsa_kv_keep(big, i32(bt), i32([4]), i32([[0, 2]]), 1, 3)
    assert bad_count() == 0 and new.tolist() == [3]
    assert torch.equal(big[N - 4:], rows[[0, 1, 3, 3]])


# ---------------------------------------------------------------------------
# streams and graphs of the small calls, and the step as a whole
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("which", ["norm", "gradient", "tree", "keep"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_results_are_the_other_streams_memory(which, as_handle):
    """Blocks of the results' sizes, freed on the current stream behind a kernel that will yet write them: a call on
    another stream gets none of them."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    c, t = Norm(40, 300, 8, 2, 192), Tree(41, [900, 300], 8, 16)
    cache, bt, lens, keep = t.cache.clone(), i32(t.bt), i32(t.lens), i32([[0, 3, -1], [1, 4, 5]])
    pos = i32(c.pos)
    args = t.args()

    def call(**kw):
        if which == "norm":
            return dsa.dsa_qk_norm_rope(*c.x, *c.w, pos, c.freqs, eps=c.eps, **kw)
        if which == "gradient":
            return dsa.dsa_qk_norm_rope_gradient(*c.g, *c.x, *c.w, pos, c.freqs, eps=c.eps, **kw)
        if which == "tree":
            return dsa.dsa_tree_decode(*args, **kw)
        return (dsa.dsa_kv_keep(cache, bt, lens, keep, 16, 8, **kw),)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    spare = [torch.empty_like(x) for x in want for _ in range(2)]
    torch.cuda.synchronize()
    blocks = {x.data_ptr() for x in spare}
    torch.cuda._sleep(20_000_000)
    for x in spare:
        x.fill_(1)
    del spare, x
    got = call(stream=s.cuda_stream if as_handle else s)
    assert not blocks & {x.data_ptr() for x in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # captured, on a side stream of the capture too
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        first = call(stream=s)
        here.wait_stream(s)
        second = call()
    for _ in range(3):
        for x in first + second:
            x.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        for a, b, w in zip(first, second, want):
            assert torch.equal(a, w) and torch.equal(b, w)


@pytest.mark.parametrize("fmt", FMTS)
def test_draft_step(fmt):
    """Three steps of four requests in one captured graph: the drafted tokens' latent rows and queries normed and turned
    by depth, appended, the tree attended, the accepted path kept.  Each attention against the oracle over what the cache
    holds; after the last step, decoding over the kept rows equals the oracle over the accepted tokens' rows in order."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(50)
    B, n, H, bs = 4, 6, 16, 16
    lens = np.array([130, 15, 400, 1], dtype=np.int32)
    bt, N = table_of(rng, lens + 4 * n, bs)
    fr, f = dsa.dsa_rope_freqs(64, layout="half", scaling="yarn", factor=4.0), O.rope_frequencies(64, 10000.0, "yarn", 4.0)
    kv = normal_bf16(rng, (N, 576))
    cache = bf(kv) if fmt == "bf16" else torch.from_numpy(O.kv_fp8_quantize(kv, 64)).cuda()
    x = torch.zeros(B * n, 1, 576, dtype=BF, device="cuda")
    qp = torch.zeros(B * n, H, 192, dtype=BF, device="cuda")
    q = torch.zeros(B, n, H, 576, dtype=BF, device="cuda")
    kw, qw = bf(normal_bf16(rng, (512,))), bf(normal_bf16(rng, (192,)))
    depth, slot, req = (torch.zeros(B * n, dtype=torch.int32, device="cuda") for _ in range(3))
    req.copy_(torch.arange(B, device="cuda").repeat_interleave(n))
    kvl, drafted = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    mask, keep = torch.zeros(B, n, dtype=torch.int64, device="cuda"), torch.zeros(B, n, dtype=torch.int32, device="cuda")
    btd = i32(bt)
    held = torch.empty_like(cache)

    def step():
        rows, _ = dsa.dsa_qk_norm_rope(x, None, kw, None, depth, fr, d_norm=512)
        turned, _ = dsa.dsa_qk_norm_rope(qp, None, qw, None, depth, fr)
        q.view(B * n, H, 576)[..., 512:].copy_(turned[..., 128:])
        dsa.dsa_kv_append(rows[:, 0, :512], rows[:, 0, 512:], slot, btd, bs, cache, token_req=req)
        out = dsa.dsa_tree_decode(q, cache, btd, kvl, mask, bs, 192 ** -0.5, num_draft=drafted)
        held.copy_(cache)
        return (*out, rows, turned, dsa.dsa_kv_keep(cache, btd, kvl, keep, bs, n, num_draft=drafted))
    slot.fill_(-1)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse, rows, turned, new = step()
    accepted = [[int(bt[b, p // bs]) * bs + p % bs for p in range(lens[b])] for b in range(B)]
    order = None   # the rows, as bits, that the accepted tokens of each request had
    first = cache.clone()
    order = [[first[r].clone() for r in rr] for rr in accepted]
    t = Tree(51, [n], n, H, bs=bs)
    for it in range(3):
        nd = np.array([n, 3, 1 + it, n], dtype=np.int32)
        words, paths, at, dep = [], [], np.full((B, n), -1), np.zeros((B, n))
        for b in range(B):
            parent = [int(rng.integers(-1, j)) if j else -1 for j in range(n)]
            words.append(ancestors(parent))
            leaf = int(rng.integers(0, nd[b]))
            path = [j for j in range(nd[b]) if words[b][leaf] >> j & 1]
            if b == 3 and it == 1:
                path = []                                                    # nothing was accepted
            paths.append(path)
            at[b, :nd[b]] = lens[b] + np.arange(nd[b])
            dep[b] = [lens[b] + bin(w).count("1") - 1 for w in words[b]]
        xb, qb, qn = normal_bf16(rng, (B * n, 1, 576)), normal_bf16(rng, (B * n, H, 192)), normal_bf16(rng, (B, n, H, 512))
        x.copy_(bf(xb)), qp.copy_(bf(qb)), q[..., :512].copy_(bf(qn))
        slot.copy_(i32(at.reshape(-1))), depth.copy_(i32(dep.reshape(-1)))
        total = (lens + nd).astype(np.int32)
        kvl.copy_(i32(total)), drafted.copy_(i32(nd)), mask.copy_(torch.from_numpy(signed(words)))
        keep.copy_(i32(np.array([p + [-1] * (n - len(p)) for p in paths])))
        g.replay()
        torch.cuda.synchronize()
        # norms
        c = Norm(1, 1, 1, 0, 576, 512, 64, "half", eps=1e-6, mscale=1.0)
        c.x, c.w, c.pos, c.f = [bf(xb), None], [kw, None], dep.reshape(-1), f
        c.check_forward((rows, None))
        c.d = c.d_norm = 192
        c.x, c.w = [bf(qb), None], [qw, None]
        c.check_forward((turned, None))
        # attention over what the cache held
        values = O.bf16_to_f64(bits(held)) if fmt == "bf16" else O.bf16_to_f64(O.kv_fp8_dequantize(held.cpu().numpy(), 64))
        t.q, t.values, t.bt, t.lens, t.mask, t.drafted, t.scale = bits(q), values, bt, total, signed(words), nd, 192 ** -0.5
        t.check((out, lse))
        # the path's rows, in order, behind the context
        for b, path in enumerate(paths):
            order[b] += [held[int(bt[b, (lens[b] + j) // bs]) * bs + (lens[b] + j) % bs].clone() for j in path]
        lens = np.array([m + len(p) for m, p in zip(lens, paths)], dtype=np.int32)
        assert np.array_equal(new.cpu().numpy(), lens)
        for b in range(B):
            at_now = [int(bt[b, p // bs]) * bs + p % bs for p in range(lens[b])]
            assert torch.equal(cache[at_now], torch.stack(order[b]))
    # the accepted tokens attended one at a time over the kept rows: a chain is decode over its prefix
    q1 = bf(normal_bf16(rng, (B, 1, H, 576)))
    one = torch.ones(B, 1, dtype=torch.int64, device="cuda")
    got = dsa.dsa_tree_decode(q1, cache, btd, i32(lens), one, bs, 0.07)
    want = dsa.dsa_paged_decode(q1[:, 0], cache, btd, i32(lens), bs, 0.07)
    assert torch.equal(got[0][:, 0], want[0]) and torch.equal(got[1][:, 0], want[1])


def test_draft_chain_equals_decode_steps():
    """A chain of drafted tokens attended at once against the same tokens attended one after another: the same keys and
    weights, summed in other tiles, so both lie within the same bound of the oracle."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    n = 5
    t = Tree(60, [300, 1029, 64], n, 16, mask=[ancestors(range(-1, n - 1))] * 3)
    t.check(t.run())
    q, cache, bt, lens, _, bs, scale = t.args()
    for i in range(n):
        out, lse = dsa.dsa_paged_decode(q[:, i].contiguous(), cache, bt, lens - (n - 1 - i), bs, scale)
        ref = O.paged_decode(t.q[:, i], t.values, t.bt, t.lens - (n - 1 - i), bs, scale)
        assert np.abs(f32(out) - ref["out"]).max() < 2 * (2.0 ** -7) * ref["spread"].max()
    assert bad_count() == 0


def test_norm_in_a_callers_autograd_function():
    import dsa_sparse_mla_prefill_gb300 as dsa
    c = Norm(70, 64, 4, 2, 128, None, 64, "half", F32)
    pos = i32(c.pos)

    class Fn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, qw, kw):
            ctx.save_for_backward(q, k, qw, kw)
            return dsa.dsa_qk_norm_rope(q, k, qw, kw, pos, c.freqs, eps=c.eps)

        @staticmethod
        def backward(ctx, gq, gk):
            q, k, qw, kw = ctx.saved_tensors
            return dsa.dsa_qk_norm_rope_gradient(gq, gk, q, k, qw, kw, pos, c.freqs, eps=c.eps)
    leaves = [t.clone().requires_grad_() for t in (*c.x, *c.w)]
    q, k = Fn.apply(*leaves)
    torch.autograd.backward([q, k], c.g)
    c.check_gradient([t.grad for t in leaves])
