"""Norms in front of the rotation and the step that checks drafted tokens, without a
GPU: the oracle against closed forms, differences and its older functions, and
every refusal of the entry points."""
import ctypes
import math

import numpy as np
import pytest

import dsa_sparse_mla_prefill_gb300 as dsa
import oracle.dsa_oracle as O
from synth import normal_bf16


@pytest.fixture(scope="module")
def lib():
    from dsa_sparse_mla_prefill_gb300 import build as b
    b.build()
    return dsa.lib()


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------
def test_norm_oracle_by_hand():
    x = np.array([[[3.0, 4.0, 7.0, 9.0]]])
    # rms of (3, 4) is 5 / sqrt 2; a quarter turn takes (a, b) to (-b, a)
    y = O.norm_rope(x, [2.0, 1.0], [1], [math.pi / 2], "half", 0.0, 2)
    s = math.sqrt(2.0) / 5
    assert np.allclose(y, [[[6 * s, 4 * s, -9, 7]]])
    # a norm of everything: the scale of x does not matter, its sign does
    w = np.arange(1.0, 5.0)
    a, b = O.norm_rope(x, w, None, None, "half", 0.0, 4), O.norm_rope(-1e3 * x, w, None, None, "half", 0.0, 4)
    assert np.allclose(a, -b) and np.isclose(((a / w) ** 2).mean(), 1.0)
    # eps is added to the mean of squares
    assert np.allclose(O.norm_rope(0 * x + 1, w, None, None, "half", 3.0, 4), w / 2)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d,d_norm,d_rope", [(8, 8, 4), (8, 4, 4), (6, 5, 4), (4, 4, 0), (4, 1, 4)])
def test_norm_gradient_oracle_is_the_difference_quotient(layout, d, d_norm, d_rope):
    rng = np.random.default_rng(d + d_norm)
    x, g = rng.standard_normal((2, 3, 2, d))
    w, pos = rng.standard_normal(d_norm), np.array([0, 5, 70])
    f = O.rope_frequencies(d_rope, 100.0) if d_rope else None
    args = (pos, f, layout, 0.01, d_norm, 1.3)

    def loss(x, w):
        return (g * O.norm_rope(x, w, *args)).sum()
    gx, gw = O.norm_rope_gradient(g, x, w, *args)
    h = 1e-6
    for grad, arr, at in ((gx, x, lambda a: loss(a, w)), (gw, w, lambda a: loss(x, a))):
        for i in np.ndindex(arr.shape):
            up, down = arr.copy(), arr.copy()
            up[i] += h
            down[i] -= h
            # (second differences of the loss are below 1e3: an error of h^2 1e3 / 6, and rounding 1e-14 / h)
            assert abs((at(up) - at(down)) / (2 * h) - grad[i]) < 1e-7


def test_tree_oracle_of_a_chain_is_decoding_token_by_token():
    rng = np.random.default_rng(3)
    B, n, H, bs, lens = 2, 3, 2, 4, [9, 3]
    kv = O.bf16_to_f64(normal_bf16(rng, (40, 576)))
    bt = np.array([[5, 2, 8], [0, 9, 1]], dtype=np.int32)
    q = normal_bf16(rng, (B, n, H, 576))
    chain = np.array([[0b1, 0b11, 0b111]] * B, dtype=np.int64)
    got = O.tree_decode(q, kv, bt, lens, chain, bs, 0.1)
    for i in range(n):
        want = O.paged_decode(q[:, i], kv, bt, [x - n + 1 + i for x in lens], bs, 0.1)
        assert np.allclose(got["out"][:, i], want["out"]) and np.allclose(got["lse"][:, i], want["lse"])
    # siblings do not see each other; a token without itself or a context sees nothing; padding
    fork = np.array([[0b1, 0b10, 0b101], [0b1, 0b0, 0b111]], dtype=np.int64)
    got = O.tree_decode(q, kv, bt, lens, fork, bs, 0.1, num_draft=[3, 2])
    keys = [bt[0, p // bs] * bs + p % bs for p in (0, 1, 2, 3, 4, 5, 7)]
    out, lse = O.attend(O.bf16_to_f64(q)[0, 1], kv[keys], kv[keys, :512], 0.1)
    assert np.allclose(got["out"][0, 1], out) and np.allclose(got["lse"][0, 1], lse)
    assert np.isneginf(got["lse"][1, 2]).all() and np.isfinite(got["lse"][1, :2]).all()


def test_keep_oracle():
    bt = np.array([[3, 0], [1, 2]])
    moves, lens, bad = O.kv_keep(bt, [6, 7], [[0, 2, 3], [1, -1, 0]], 4, 16, 4)
    # request 0: context 2, tokens at 2..5; token 2 (position 4, page 0) to position 3, token 3 to 4
    assert moves == [(0, 15), (1, 0), (8, 7)] and lens.tolist() == [5, 4] and bad == 0
    moves, lens, bad = O.kv_keep(bt, [6, 7], [[1, 1, 3], [4, -1, 0]], 4, 16, 4)
    assert moves == [(15, 14)] and lens.tolist() == [3, 3] and bad == 2
    moves, lens, bad = O.kv_keep(bt, [0, 3], [[1], [1]], 4, 16, 4)      # padding; more drafted than there are positions
    assert moves == [] and lens.tolist() == [0, 3] and bad == 1


# ---------------------------------------------------------------------------
# refusals: none of these reaches the GPU
# ---------------------------------------------------------------------------
def _vp(x=4096):
    return ctypes.c_void_p(x)


INVALID, UNSUPPORTED, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK
WS = 64 << 20

NORM = [
    (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(wd=2), UNSUPPORTED), (dict(d=0), INVALID), (dict(dn=0), INVALID), (dict(dn=193), INVALID), (dict(d=2048, dn=2048), UNSUPPORTED),
    (dict(d=63, dn=63), INVALID),                                   # less than the columns to turn
    (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(Hq=0, Hk=0, q=None, k=None), OK), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qo=None), INVALID),
    (dict(qw=None), INVALID), (dict(kw=None), INVALID), (dict(kw=4097), INVALID), (dict(wd=1, qw=4098), INVALID),
    (dict(pos=None), INVALID), (dict(pos=4098), INVALID), (dict(q=4097), INVALID), (dict(dtype=1, k=4098), INVALID),
    (dict(qt=-8), INVALID), (dict(ko=1 << 21), INVALID),            # the two results in one place
    (dict(T=1 << 20, Hq=4096), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", NORM + [
    (dict(T=0, q=None, k=None), OK), (dict(qos=191), INVALID), (dict(qot=4 * 192 - 1), INVALID), (dict(qos=0), INVALID),
    (dict(q=1 << 21, qs=384), INVALID)])                            # in place with other strides
def test_norm_refusals(lib, change, want):
    a = dict(dict(q=4096, qt=4 * 192, qs=192, qo=1 << 21, qot=4 * 192, qos=192, Hq=4, k=8192, ko=1 << 22, Hk=2, dtype=0, qw=4096,
                  kw=4096, wd=0, pos=4096, T=10, d=192, dn=192, eps=1e-6), **change)
    f = dsa.dsa_rope_freqs(64)
    assert lib.dsa_qk_norm_rope(_vp(a["q"]), a["qt"], a["qs"], _vp(a["qo"]), a["qot"], a["qos"], a["Hq"], _vp(a["k"]), 384, 192,
                                _vp(a["ko"]), 384, 192, a["Hk"], a["dtype"], _vp(a["qw"]), _vp(a["kw"]), a["wd"], _vp(a["pos"]),
                                a["T"], a["d"], a["dn"], a["eps"], ctypes.byref(f), None) == want


@pytest.mark.parametrize("change,want", NORM + [
    (dict(g=None), INVALID), (dict(g=4097), INVALID), (dict(gt=-192), INVALID), (dict(g=1 << 21), INVALID),
    (dict(q=1 << 21), INVALID), (dict(dw=None), INVALID), (dict(dw=4098), INVALID), (dict(dk=4096), INVALID),
    (dict(ws=None), INVALID), (dict(ws=4100), INVALID), (dict(wsb=304 * 192 * 4 - 1), INVALID)])
def test_norm_gradient_refusals(lib, change, want):
    a = dict(dict(g=16384, gt=4 * 192, q=4096, qt=4 * 192, qo=1 << 21, Hq=4, k=8192, ko=1 << 22, Hk=2, dtype=0, qw=4096, kw=4096,
                  wd=0, pos=4096, T=10, d=192, dn=192, eps=1e-6, dw=4096, dk=8192, ws=4096, wsb=WS), **change)
    f = dsa.dsa_rope_freqs(64)
    assert lib.dsa_qk_norm_rope_gradient(
        _vp(a["g"]), a["gt"], 192, _vp(a["q"]), a["qt"], 192, _vp(a["qo"]), a["Hq"], _vp(32768), 384, 192, _vp(a["k"]), 384,
        192, _vp(a["ko"]), a["Hk"], a["dtype"], _vp(a["qw"]), _vp(a["kw"]), a["wd"], _vp(a["pos"]), a["T"], a["d"], a["dn"],
        a["eps"], ctypes.byref(f), _vp(a["dw"]), _vp(a["dk"]), _vp(a["ws"]), a["wsb"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), INVALID), (dict(B=0, q=None, ws=None, mask=None), OK), (dict(n=0), UNSUPPORTED), (dict(n=65), UNSUPPORTED),
    (dict(n=-1), INVALID), (dict(H=0), UNSUPPORTED), (dict(H=129), UNSUPPORTED), (dict(n=33, H=64), UNSUPPORTED),
    (dict(dqk=544), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(fmt=7), UNSUPPORTED), (dict(ld_kv=568), INVALID),
    (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(N=-1), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(mask=None), INVALID), (dict(mask=4100), INVALID), (dict(nd=4098), INVALID), (dict(out=None), INVALID),
    (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(ws=4096 + 128), INVALID), (dict(wsb=100000), INVALID),
    (dict(q=4104), INVALID), (dict(out=4104), INVALID), (dict(B=1 << 25, H=32, n=64), UNSUPPORTED)])
def test_tree_refusals(lib, change, want):
    a = dict(dict(q=4096, cache=4096, fmt=0, N=100, ld_kv=576, bt=4096, mb=4, bs=16, lens=4096, mask=4096, nd=None, B=2, n=4,
                  H=16, dqk=576, dv=512, scale=0.1, out=4096, lse=4096, ws=4096, wsb=WS), **change)
    assert lib.dsa_tree_decode(_vp(a["q"]), _vp(a["cache"]), a["fmt"], a["N"], a["ld_kv"], _vp(a["bt"]), a["mb"], a["bs"],
                               _vp(a["lens"]), _vp(a["mask"]), _vp(a["nd"]), a["B"], a["n"], a["H"], a["dqk"], a["dv"],
                               a["scale"], _vp(a["out"]), _vp(a["lse"]), _vp(a["ws"]), a["wsb"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(num=0), INVALID), (dict(num=129), UNSUPPORTED), (dict(caches=None), INVALID), (dict(first=None), INVALID),
    (dict(first=4104), INVALID), (dict(first=1 << 22), INVALID),    # the same cache twice
    (dict(first=(1 << 22) - 99 * 1152), INVALID), (dict(first=(1 << 22) + 99 * 1152), INVALID),   # one reaching into the other
    (dict(rb=1150), INVALID), (dict(rb=0), INVALID), (dict(rb=1 << 25), UNSUPPORTED), (dict(N=-1), INVALID), (dict(mb=0), INVALID),
    (dict(bs=0), INVALID), (dict(n=-1), INVALID), (dict(n=65), UNSUPPORTED), (dict(m=-1), INVALID), (dict(m=65), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(B=0, bt=None), OK), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(keep=None), INVALID), (dict(new=None), INVALID), (dict(new=4096), INVALID),   # the lengths in place
    (dict(new=4100), INVALID), (dict(nd=8196), INVALID), (dict(keep=8192 - 28), INVALID), (dict(bt=8192 - 28), INVALID),
    (dict(bt=4098), INVALID), (dict(lens=4097), INVALID), (dict(nd=4097), INVALID), (dict(keep=4098), INVALID),
    (dict(new=8194), INVALID)])
def test_keep_refusals(lib, change, want):
    a = dict(dict(caches=1, first=4096, num=2, rb=1152, N=100, bt=4096, mb=4, bs=16, lens=4096, nd=None, n=8, keep=4096, m=4, B=2,
                  new=8192), **change)
    arr = (ctypes.c_void_p * 130)(*([a["first"], 1 << 22] + [(1 << 23) * (i + 1) for i in range(128)]))
    assert lib.dsa_kv_keep(arr if a["caches"] else None, a["num"], a["rb"], a["N"], _vp(a["bt"]), a["mb"], a["bs"],
                           _vp(a["lens"]), _vp(a["nd"]), a["n"], _vp(a["keep"]), a["m"], a["B"], _vp(a["new"]), None) == want


def test_workspace_sizes(lib):
    for n, H in [(1, 16), (8, 16), (4, 128), (64, 32), (3, 5)]:
        for B, positions in [(1, 1), (4, 777), (3, 100000), (0, 5)]:
            most = dsa.dsa_tree_decode_workspace(B, n, H, positions)
            assert most > 0
            if n * H <= 32:   # (the decode kernel's split; more rows are cut in tiles of 256 keys for CTA pairs)
                assert most == dsa.dsa_paged_decode_workspace(B, n * H, positions)
    for bad in [(-1, 4, 16, 1), (1, 0, 16, 1), (1, 65, 16, 1), (1, 4, 0, 1), (1, 4, 129, 1), (1, 33, 64, 1), (1, 4, 16, -1)]:
        with pytest.raises(dsa.DSAError):
            dsa.dsa_tree_decode_workspace(*bad)
    assert dsa.dsa_qk_norm_rope_gradient_workspace(192) == 304 * 192 * 4
    for bad in (0, -1, 1025):
        with pytest.raises(dsa.DSAError):
            dsa.dsa_qk_norm_rope_gradient_workspace(bad)


def test_binding_refuses_before_the_library(lib):
    import torch
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    w, pos = torch.ones(64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(None, None, None, None, pos)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope(x, None, w, None, pos)                  # host tensor
    with pytest.raises(TypeError):
        dsa.dsa_qk_norm_rope(x.half(), None, w, None, pos)
    with pytest.raises(TypeError):
        dsa.dsa_qk_norm_rope(x, None, w, None, pos, freqs=64)
    with pytest.raises(ValueError):
        dsa.dsa_qk_norm_rope_gradient(x, None, x, None, w, None, pos)
    with pytest.raises(ValueError):
        dsa.dsa_tree_decode(x[None], x, pos, pos, pos, 16, 1.0)
    with pytest.raises(TypeError):
        dsa.dsa_tree_decode(x[None].float(), x, pos, pos, pos, 16, 1.0)
    with pytest.raises(ValueError):
        dsa.dsa_kv_keep([], pos, pos, pos, 16, 4)
    with pytest.raises(ValueError):
        dsa.dsa_kv_keep(x[0], pos, pos, pos, 16, 4)
    with pytest.raises(TypeError):
        dsa.dsa_kv_keep(x[0].float(), pos, pos, pos, 16, 4)


@pytest.mark.parametrize("tiles,groups", [([7], 76), ([1, 1, 1], 76), ([400], 76), ([3, 0, 0, 9, 1, 1, 40], 9), ([1] * 300, 76),
                                          ([2, 1] * 90, 38), ([0, 0, 5], 2), ([17, 64, 30, 128, 90, 44, 23, 50], 19), ([2 ** 25, 3, 2 ** 29], 76)])
def test_split_with_blank_tiles(tiles, groups):
    """The pair form's split, a blank tile in front of every request: what a range holds, written down tile by tile,
    against the border that the joining kernel takes from its end (request, first range, parts, and whether the
    request is the first one of its first range)."""
    import ctypes
    import os
    import dsa_sparse_mla_prefill_gb300 as dsa
    from dsa_sparse_mla_prefill_gb300 import build
    build.build()
    lib = ctypes.CDLL(os.path.join(os.path.dirname(dsa.__file__), "libdsa_selftest.so"))
    u, i = ctypes.c_uint, ctypes.c_int
    total, ng = sum(n + 1 for n in tiles if n), min(sum(tiles), groups)
    begin = [g * total // ng for g in range(ng + 1)]
    held = [[] for _ in range(ng)]            # of each range: (request, first tile, behind the last)
    at = 0
    for b, n in enumerate(tiles):
        if n == 0:
            continue
        at += 1
        for g in range(ng):
            lo, hi = max(begin[g], at), min(begin[g + 1], at + n)
            if lo < hi:
                held[g].append((b, lo - at, hi - at))
        at += n
    assert sum(hi - lo for h in held for _, lo, hi in h) == sum(tiles)
    cuts = 0
    for g in range(ng):
        cut = (ctypes.c_int * 4)()
        b, _, hi = held[g][-1] if held[g] else (0, 0, 0)
        got = lib.dsa_selftest_border_gap(u(total), u(ng), u(1), i(b), i(tiles[b] if held[g] else 0), i(hi), u(g), i(len(tiles)),
                                          i(groups), cut)
        if hi == tiles[b] or not held[g]:
            assert not got
            continue
        of = [x for x in range(ng) if any(s[0] == b for s in held[x])]
        assert got and of == list(range(of[0], of[-1] + 1))
        assert tuple(cut) == (b, of[0], len(of), int(held[of[0]][0][0] == b))
        cuts += 1
    assert cuts > 0 or max(tiles) < 3
