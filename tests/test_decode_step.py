"""The decode step without a GPU: the oracle's rotary positions, cache append
and paged attention against closed forms and against the oracle's older
functions, the frequency table, and every refusal of the entry points."""
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
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_oracle_is_a_rotation(layout):
    rng = np.random.default_rng(1)
    d, T = 16, 5
    f = O.rope_frequencies(d, 10000.0)
    x, g = rng.standard_normal((2, T, 3, d))
    pos = np.array([0, 1, 7, 1000, 123456])
    y = O.rope(x, pos, f, layout, 1.25)
    assert np.allclose(y[0], 1.25 * x[0], atol=1e-15)               # position 0 only scales
    assert np.allclose((y ** 2).sum(-1), 1.25 ** 2 * (x ** 2).sum(-1))
    # the gradient is the transpose: <g, R x> = <R^T g, x>
    assert np.isclose((g * y).sum(), (O.rope(g, pos, f, layout, 1.25, gradient=True) * x).sum())
    # scores depend on the distance alone
    a = O.rope(x[:1], [40], f, layout) @ O.rope(g[:1], [33], f, layout).transpose(0, 2, 1)
    b = O.rope(x[:1], [7], f, layout) @ O.rope(g[:1], [0], f, layout).transpose(0, 2, 1)
    assert np.allclose(a, b)


def test_rope_oracle_pairs_by_hand():
    # one turn of 90 degrees per position: (a, b) -> (-b, a)
    x = np.arange(1.0, 5.0)[None]
    assert np.allclose(O.rope(x, [1], [math.pi / 2] * 2, "interleaved"), [[-2, 1, -4, 3]])
    assert np.allclose(O.rope(x, [1], [math.pi / 2] * 2, "half"), [[-3, -4, 1, 2]])


def test_yarn_oracle_ends():
    d, base, L, s = 64, 10000.0, 4096, 40.0
    f, y = O.rope_frequencies(d, base), O.rope_frequencies(d, base, "yarn", s, L, 32.0, 1.0)
    turns = f * L / (2 * math.pi)
    assert np.allclose(y[turns > 32 * 2], f[turns > 32 * 2])        # fast pairs are kept
    assert np.allclose(y[turns < 0.5], f[turns < 0.5] / s)          # slow ones interpolated
    assert np.all(y <= f * (1 + 1e-15)) and np.all(y >= f / s * (1 - 1e-15))
    assert np.all(np.diff(y) < 0)


def test_paged_decode_oracle_equals_sparse_prefill():
    rng = np.random.default_rng(3)
    B, H, bs, lens = 3, 2, 4, [9, 0, 16]
    kv = normal_bf16(rng, (40, 576))
    bt = np.array([[5, 2, 8, -1], [-1] * 4, [0, 9, 1, 7]], dtype=np.int32)
    q = normal_bf16(rng, (B, H, 576))
    idx = np.full((B, 16), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        idx[b, :n] = [bt[b, p // bs] * bs + p % bs for p in range(n)]
    want, lse = O.sparse_prefill(q, kv, idx, 16, 0.1, 576, 512)
    got = O.paged_decode(q, O.bf16_to_f64(kv), bt, lens, bs, 0.1)
    assert np.allclose(got["out"], want) and np.allclose(got["lse"][[0, 2]], lse[[0, 2]]) and got["bad"] == 0
    assert np.all(np.isneginf(got["lse"][1]))
    # its own positions, some absent, some bad (past the length, unmapped block)
    sel = np.array([[3, -1, 8, 9, -5], [0, 1, -1, -1, -1], [15, 2, -1, -1, 7]], dtype=np.int32)
    loc = np.full((B, 5), -1, dtype=np.int32)
    for b in range(B):
        for e, p in enumerate(sel[b]):
            if 0 <= p < lens[b]:
                loc[b, e] = bt[b, p // bs] * bs + p % bs
    want, lse = O.sparse_prefill(q, kv, loc, 5, 0.1, 576, 512)
    got = O.paged_decode(q, O.bf16_to_f64(kv), bt, lens, bs, 0.1, idx=sel, k=5)
    assert np.allclose(got["out"], want) and got["bad"] == 2        # (request 1 has no keys: nothing is looked at)


def test_append_rows_oracle():
    bt = np.array([[3, -1], [0, 7]])
    rows, bad = O.append_rows([0, 5, 4, -1, -2, 8, 3], [0, 1, 0, 9, 0, 1, 2], bt, 4, 31)
    assert rows.tolist() == [12, 29, -1, -1, -1, -1, -1] and bad == 4
    rows, bad = O.append_rows([1, 7], None, bt, 4, 31)
    assert rows.tolist() == [13, -1] and bad == 1                    # row 31 is outside the cache


# ---------------------------------------------------------------------------
# frequency table
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [2, 32, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("yarn", 40.0), ("yarn", 1.0), ("linear", 0.5)])
def test_frequency_table(lib, d, scaling, factor):
    f = dsa.dsa_rope_freqs(d, base=50000.0, layout="half", scaling=scaling, factor=factor, mscale=1.5)
    want = O.rope_frequencies(d, 50000.0, scaling, factor) / (2 * math.pi)
    got = np.array([f.turns[i] / 2.0 ** 64 for i in range(d // 2)])
    # the table holds doubles: f has a few roundings of 2^-53, relative to a value below 1
    assert np.abs(got - want % 1.0).max() <= 16 * 2.0 ** -53
    assert f.d_rope == d and f.layout == 1 and f.mscale == 1.5
    assert all(f.turns[i] == 0 for i in range(d // 2, 128))


# ---------------------------------------------------------------------------
# refusals: none of these reaches the GPU
# ---------------------------------------------------------------------------
def _vp(x=4096):
    return ctypes.c_void_p(x)


INVALID, UNSUPPORTED, OK = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_OK


@pytest.mark.parametrize("change,want", [
    (dict(d=0), INVALID), (dict(d=63), INVALID), (dict(d=258), UNSUPPORTED), (dict(base=0.5), INVALID),
    (dict(base=math.inf), INVALID), (dict(base=1.0), OK), (dict(base=1.0, scaling=2), INVALID), (dict(layout=2), INVALID),
    (dict(scaling=3), INVALID), (dict(factor=0.0), INVALID), (dict(factor=math.nan), INVALID),
    (dict(scaling=2, L=0), INVALID), (dict(scaling=2, slow=0.0), INVALID), (dict(scaling=2, fast=0.5), INVALID),
    (dict(mscale=math.nan), INVALID), (dict(scaling=2), OK)])
def test_freqs_refusals(lib, change, want):
    a = dict(dict(d=64, base=10000.0, layout=0, scaling=0, factor=2.0, L=4096, fast=32.0, slow=1.0, mscale=1.0), **change)
    f = dsa.RopeFreqs()
    assert lib.dsa_rope_freqs_init(ctypes.byref(f), a["d"], a["base"], a["layout"], a["scaling"], a["factor"], a["L"],
                                   a["fast"], a["slow"], a["mscale"]) == want
    assert lib.dsa_rope_freqs_init(None, 64, 1e4, 0, 0, 1.0, 4096, 32.0, 1.0, 1.0) == INVALID


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(H=-1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(T=0, x=None), OK),
    (dict(H=0, y=None), OK), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID),
    (dict(x=4097), INVALID), (dict(y=4097), INVALID), (dict(pos=4098), INVALID), (dict(dtype=1, x=4098), INVALID),
    (dict(yh=63), INVALID), (dict(yt=4 * 64 - 1), INVALID), (dict(yt=64, yh=64 * 9), INVALID),
    (dict(yh=0), INVALID), (dict(yt=0), INVALID), (dict(xt=-64), INVALID),
    (dict(x=8192, y=8192, xh=64, yh=128, yt=1024, xt=1024), INVALID)])
def test_rope_refusals(lib, change, want):
    a = dict(dict(x=4096, xt=4 * 64, xh=64, y=1 << 20, yt=4 * 64, yh=64, dtype=0, pos=4096, T=10, H=4), **change)
    f = dsa.dsa_rope_freqs(64)
    assert lib.dsa_rope(_vp(a["x"]), a["xt"], a["xh"], _vp(a["y"]), a["yt"], a["yh"], a["dtype"], _vp(a["pos"]), a["T"],
                        a["H"], ctypes.byref(f), 0, None) == want
    assert lib.dsa_rope(_vp(), 64, 64, _vp(1 << 20), 64, 64, 0, _vp(), 1, 1, None, 0, None) == INVALID


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(T=0, c=None), OK), (dict(dr=32), UNSUPPORTED), (dict(fmt=2), UNSUPPORTED),
    (dict(dr=0), UNSUPPORTED),                                       # frequencies of another width
    (dict(ld=568), INVALID), (dict(ld=580), INVALID), (dict(cs=516), INVALID), (dict(cs=256), INVALID),
    (dict(ps=32), INVALID), (dict(ps=68), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID),
    (dict(N=-1), INVALID), (dict(nreq=9, req=None), INVALID),        # more tokens than requests
    (dict(nreq=-1), INVALID), (dict(c=None), INVALID), (dict(pe=None), INVALID), (dict(pos=None), INVALID),
    (dict(bt=None), INVALID), (dict(cache=None), INVALID), (dict(c=4104), INVALID), (dict(pe=4104), INVALID),
    (dict(cache=4104), INVALID), (dict(req=4097), INVALID), (dict(bt=4098), INVALID), (dict(pos=4098), INVALID)])
def test_append_refusals(lib, change, want):
    a = dict(dict(c=4096, cs=512, pe=4096, ps=64, T=10, dr=64, pos=4096, req=4096, bt=4096, nreq=3, mb=4, bs=16,
                  cache=4096, fmt=0, N=100, ld=576), **change)
    f = dsa.dsa_rope_freqs(64)
    assert lib.dsa_kv_append(_vp(a["c"]), a["cs"], _vp(a["pe"]), a["ps"], a["T"], a["dr"], _vp(a["pos"]),
                             _vp(a["req"]), _vp(a["bt"]), a["nreq"], a["mb"], a["bs"], ctypes.byref(f), _vp(a["cache"]),
                             a["fmt"], a["N"], a["ld"], None) == want


WS = 64 << 20


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), INVALID), (dict(B=0, q=None, ws=None), OK), (dict(H=0), UNSUPPORTED), (dict(H=129), UNSUPPORTED),
    (dict(dqk=544), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(fmt=7), UNSUPPORTED), (dict(ld_kv=568), INVALID),
    (dict(ld_kv=580), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(N=-1), INVALID),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=-3e38), INVALID), (dict(k=9), INVALID), (dict(k=-1), INVALID),
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(ws=4096 + 128), INVALID),
    (dict(wsb=100000), INVALID), (dict(q=4104), INVALID), (dict(cache=4104), INVALID), (dict(out=4104), INVALID),
    (dict(idx=4098), INVALID), (dict(lens=4097), INVALID), (dict(bt=4098), INVALID), (dict(lse=4098), INVALID),
    (dict(B=1 << 25, H=128), UNSUPPORTED), (dict(B=1 << 20, mb=1 << 20, bs=1 << 10, H=1, idx=None), UNSUPPORTED)])
def test_decode_refusals(lib, change, want):
    a = dict(dict(q=4096, cache=4096, fmt=0, N=100, ld_kv=576, bt=4096, mb=4, bs=16, lens=4096, idx=4096, k=8, ld=8, B=2,
                  H=16, dqk=576, dv=512, scale=0.1, out=4096, lse=4096, ws=4096, wsb=WS), **change)
    assert lib.dsa_paged_decode(_vp(a["q"]), _vp(a["cache"]), a["fmt"], a["N"], a["ld_kv"], _vp(a["bt"]), a["mb"],
                                a["bs"], _vp(a["lens"]), _vp(a["idx"]), a["k"], a["ld"], a["B"], a["H"], a["dqk"],
                                a["dv"], a["scale"], _vp(a["out"]), _vp(a["lse"]), _vp(a["ws"]), a["wsb"], None) == want


def test_workspace_sizes(lib):
    # two partial results per range, all heads padded to whole head blocks, plus their log-sum-exp and a
    # little; a range per SM and head block (of 64 heads), but no more than there are tiles of 128 positions
    for H, hp, most in [(1, 16, 152), (16, 16, 152), (17, 32, 152), (32, 32, 152), (33, 64, 152), (128, 128, 76)]:
        for B, positions in [(1, 1), (1, 777), (4, 128), (3, 100000), (0, 5), (2, 0)]:
            ranges = max(1, min(most, B * -(-positions // 128)))
            need = 2 * ranges * hp * 4 * (512 + 1)
            assert need <= dsa.dsa_paged_decode_workspace(B, H, positions) < need + 4096
    for bad in [(-1, 16, 1), (1, 0, 1), (1, 129, 1), (1, 16, -1)]:
        with pytest.raises(dsa.DSAError):
            dsa.dsa_paged_decode_workspace(*bad)


def test_binding_refuses_before_the_library(lib):
    import torch
    f = dsa.dsa_rope_freqs(64)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, pos, f)                                      # host tensor
    with pytest.raises(TypeError):
        dsa.dsa_rope(x.to(torch.float16), pos, f)
    with pytest.raises(ValueError):
        dsa.dsa_rope_freqs(64, layout="pairs")
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope_freqs(63)
    with pytest.raises(TypeError):
        dsa.dsa_kv_append(x.float(), None, pos, pos, 16, x)
    with pytest.raises(ValueError):
        dsa.dsa_paged_decode(x, x, pos, pos, 16, 1.0)
