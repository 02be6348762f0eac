"""What the decode step does when something is not as it should be: the joining kernel over borders that no
call wrote, waits that run out."""
import ctypes
import os

import numpy as np
import pytest

from gpu_util import f32, need_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def selftest():
    need_gpu()
    import dsa_sparse_mla_prefill_gb300 as dsa
    return ctypes.CDLL(os.path.join(os.path.dirname(dsa.__file__), "libdsa_selftest.so"))


class Join:
    """Parts of B requests of 16 heads in a split over `groups` ranges; out and lse with rows before and behind."""

    def __init__(self, tiles, groups, seed=0):
        rng = np.random.default_rng(seed)
        self.tiles, self.groups, self.B = tiles, groups, len(tiles)
        self.total, self.ng = sum(tiles), min(sum(tiles), groups)
        self.po = rng.standard_normal((2 * groups, 16, 512)).astype(np.float32)
        self.pl = (rng.standard_normal((2 * groups, 16)) * 8).astype(np.float32)
        self.pl[rng.random((2 * groups, 16)) < 0.1] = -np.inf
        self.borders = np.zeros((1 + groups, 4), np.int32)

    def run(self, selftest, H, ten):
        p = [torch.from_numpy(x).cuda() for x in (self.borders, self.po, self.pl)]
        self.big = torch.full((self.B + 4, H, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B + 4, H), 5.0, device="cuda")
        vp = ctypes.c_void_p
        rc = selftest.dsa_selftest_join(*(vp(t.data_ptr()) for t in p), vp(self.big[2:].data_ptr()), vp(self.lse[2:].data_ptr()),
                                        self.B, H, self.groups, ten, vp(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        torch.cuda.synchronize()
        assert (self.big[:2] == 5).all() and (self.big[-2:] == 5).all()
        assert (self.lse[:2] == 5).all() and (self.lse[-2:] == 5).all()
        return self.big[2:-2], self.lse[2:-2]


@pytest.mark.parametrize("ten", [0, 1])
@pytest.mark.parametrize("tiles,groups,H", [([7], 152, 16), ([1024], 152, 9), ([3, 9, 1, 1, 40], 38, 16), ([5] * 60, 76, 1)])
def test_join_of_parts(selftest, tiles, groups, H, ten):
    """Against 64 bits: sums of up to 152 parts in float32, each addition and product half a step (2^-24) of the sum of
    magnitudes, in the weighted values and in the weights, and exp2 and log2 to 2^-21: below 2^-15 together, then the
    rounding to bf16 (2^-8)."""
    j = Join(tiles, groups, 1)
    begin = [g * j.total // j.ng for g in range(j.ng + 1)]
    starts = np.concatenate([[0], np.cumsum(tiles)])
    parts = {b: [] for b in range(j.B)}
    j.borders[0, :2] = j.total, j.ng
    for g in range(j.ng):
        for b in range(j.B):
            if starts[b] < begin[g + 1] and starts[b + 1] > begin[g]:
                whole = starts[b] >= begin[g] and starts[b + 1] <= begin[g + 1]
                parts[b] += [] if whole else [2 * g + int(starts[b] > begin[g])]
                if starts[b + 1] >= begin[g + 1]:
                    j.borders[1 + g, :3] = b, tiles[b], begin[g + 1] - starts[b]
    out, lse = j.run(selftest, H, ten)
    got, got_l = f32(out), lse.double().cpu().numpy()
    for b in range(j.B):
        if not parts[b]:
            assert (got[b] == 5).all() and (got_l[b] == 5).all()
            continue
        l, o = j.pl[parts[b], :H].astype(np.float64), j.po[parts[b], :H].astype(np.float64)
        m = l.max(0)
        none = np.isinf(m)
        w = np.exp2(l - np.where(none, 0, m))
        s = np.where(none, 1, w.sum(0))
        want, size = (np.einsum("ph,phd->hd", w, x) / s[:, None] for x in (o, np.abs(o)))
        tol = 2.0 ** -15 * size
        assert (np.abs(got[b] - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()
        assert np.array_equal(np.isneginf(got_l[b]), none)
        want_l = (np.where(none, 0, m) + np.log2(s)) * np.log(2)
        assert (np.abs(np.where(none, 0, got_l[b]) - np.where(none, 0, want_l)) <= 2.0 ** -15 + 2.0 ** -22 * np.abs(want_l)).all()


@pytest.mark.parametrize("fill", ["zeros", "ones", "bytes", "random", "near"])
def test_join_over_borders_that_no_call_wrote(selftest, fill):
    """A split whose ranges gave up before their last tile: the entries are whatever the memory held, and nothing
    outside the call's outputs is written."""
    rng = np.random.default_rng(4)
    j = Join([40, 3, 9], 38)
    n = j.borders[1:].shape
    j.borders[1:] = {"zeros": 0, "ones": -1, "bytes": 0x7f7f7f7f, "random": rng.integers(-2 ** 31, 2 ** 31, n),
                     "near": rng.integers(-3, 60, n)}[fill]
    j.borders[0, :2] = j.total, j.ng
    out, lse = j.run(selftest, 16, 0)
    if fill != "near":
        assert (out == 5).all() and (lse == 5).all()
    # ... and with a head that no call wrote either
    j.borders[0] = 0x7f7f7f7f
    out, lse = j.run(selftest, 16, 1)
    assert (out == 5).all() and (lse == 5).all()


@pytest.mark.parametrize("poll", [0, 1])
@pytest.mark.parametrize("kind", ["completes", "runs out", "another gave up"])
def test_voted_wait(selftest, poll, kind):
    """Every lane of the waiting warps gets the same answer, and a wait that runs out is counted once for its CTA."""
    import time
    got = torch.full((96,), -1, dtype=torch.int32, device="cuda")
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    vp = ctypes.c_void_p
    t0 = time.time()
    rc = selftest.dsa_selftest_wait(poll, ["completes", "runs out", "another gave up"].index(kind), ctypes.c_uint(200000),
                                    vp(got.data_ptr()), vp(err.data_ptr()), vp(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    assert got.tolist() == [int(kind == "completes")] * 96
    assert err.tolist() == [0, int(kind == "runs out"), 0, 0]
    assert (elapsed > 1.5) == (kind == "runs out") and elapsed < 60      # the wait limit is 2 s


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("page", [8, 64, 128])
def test_rows_that_are_columns_of_a_wider_buffer(selftest, H, page):
    """The last columns of a buffer, which ends with the last row's: the same bits as from rows of their own."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    torch.manual_seed(5)
    N, B, pages = 40 * 128, 3, 10 * 128 // page
    wide = torch.full((N, 1152), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 576:].normal_()
    table = torch.randperm(N // page, device="cuda")[:B * pages].to(torch.int32).reshape(B, pages).contiguous()
    table[0, -1] = N // page - 1
    lens = torch.tensor([pages * page, 700, 129], dtype=torch.int32, device="cuda")
    q = torch.randn(B, H, 576, dtype=torch.bfloat16, device="cuda")
    want = dsa.dsa_paged_decode(q, wide[:, 576:].contiguous(), table, lens, page, 0.07)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(dsa.dsa_paged_decode_workspace(B, H, pages * page), dtype=torch.uint8, device="cuda")
    rc = dsa.lib().dsa_paged_decode(q.data_ptr(), wide[:, 576:].data_ptr(), 0, N, 1152, table.data_ptr(), pages, page,
                                    lens.data_ptr(), None, 0, 0, B, H, 576, 512, 0.07, out.data_ptr(), lse.data_ptr(),
                                    ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert dsa.dsa_last_device_error()[0] == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_refused_launch_attribute_is_not_left_for_the_next_launch(selftest):
    """More shared memory than a CTA can have is refused, once: no error stays pending, and less is granted after."""
    assert selftest.dsa_selftest_allow_smem(ctypes.c_uint(1 << 20)) == 1
    assert selftest.dsa_selftest_allow_smem(ctypes.c_uint(100 << 10)) == 0
    assert selftest.dsa_selftest_allow_smem(ctypes.c_uint(100 << 10)) == 0
    torch.zeros(4, device="cuda").add_(1)
    torch.cuda.synchronize()
