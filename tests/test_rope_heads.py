"""Rotary positions: how a token's heads are dealt to threads, up to the most heads an int32 counts."""
import ctypes
import os

import numpy as np
import pytest

import dsa_sparse_mla_prefill_gb300 as dsa


@pytest.fixture(scope="module")
def lib():
    from dsa_sparse_mla_prefill_gb300 import build as b
    b.build()
    return ctypes.CDLL(os.path.join(os.path.dirname(dsa.__file__), "libdsa_selftest.so"))


@pytest.mark.parametrize("H", [1, 2, 3, 16, 24, 127, 128, 2 ** 20 + 1, 2 ** 29 + 3, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("per_group", [1, 8, 128, 16384 * 16])
def test_head_groups(lib, H, per_group):
    """Heads per thread are a power of two, the largest that leaves half of the SMs' threads; every head the kernel's
    loop looks at (four steps behind the last one at most) is counted in 32 unsigned bits."""
    groups = lib.dsa_selftest_rope_head_groups(H, ctypes.c_longlong(per_group), 152)
    each = 1
    while 2 * each <= H and -(-H // (2 * each)) * per_group >= 1024 * 152:
        each *= 2
    assert groups == -(-H // each)
    assert H + 4 * groups < 2 ** 32


@pytest.mark.gpu
def test_rope_of_the_most_heads():
    """One token of 2^31 - 1 heads of one pair, in place, against the formula on pieces of it: at most ten float32
    roundings of |a| + |b| <= 4 (10 x 2^-24 x 4 < 2^-18), then the one to bf16."""
    from gpu_util import i32, need_gpu, torch
    need_gpu()
    H = 2 ** 31 - 1
    x = torch.empty(1, H, 2, dtype=torch.bfloat16, device="cuda")          # 8.6 GB
    x[:] = 1.0
    x[0, ::3, 0] = -0.5
    x[0, -1, 1] = 3.0
    pieces = [slice(0, 1000), slice(2 ** 30 - 500, 2 ** 30 + 500), slice(H - 1000, H)]
    keep = [x[0, p].double().cpu() for p in pieces]
    total = int((x[0, :, 0] == 1).sum())
    dsa.dsa_rope(x, i32([12345]), dsa.dsa_rope_freqs(2), out=x)
    torch.cuda.synchronize()
    assert dsa.dsa_last_device_error()[0] == 0
    c, s = np.cos(12345.0), np.sin(12345.0)                                # (the one frequency is 1)
    for p, k in zip(pieces, keep):
        want = torch.stack([k[:, 0] * c - k[:, 1] * s, k[:, 0] * s + k[:, 1] * c], 1)
        assert ((x[0, p].double().cpu() - want).abs() <= 2.0 ** -18 + 2.0 ** -8 * (want.abs() + 2.0 ** -18)).all()
    one = x[0, 1]                                                          # what (1, 1) was turned into, everywhere
    assert int((x[0, :, 0] == one[0]).sum()) == total                      # (the last head's first element was -0.5)
    with pytest.raises(dsa.DSAError):
        dsa.dsa_rope(x.reshape(-1)[:2].expand(1, 2 ** 31, 2), i32([0]), dsa.dsa_rope_freqs(2), out=x[:, :1].expand(1, 2 ** 31, 2))
