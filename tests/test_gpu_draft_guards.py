"""The step that checks drafted tokens, where its kernels and calls could go wrong in
ways that random inputs do not show.  GPU, against the 64-bit oracle or exact values.

Tolerances are those of test_gpu_draft_step.py, or exact; the others are derived where
they stand.  u = 2^-24, half a step of float32.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle.dsa_oracle as O
from gpu_util import bf, f32, i32, need_gpu, torch
from test_gpu_draft_step import BF, F32, U, Norm, Tree, ancestors, bad_count, f64, signed

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(3, 16), (7, 16), (8, 32)])
@pytest.mark.parametrize("per_range", [2, 3, 5])
def test_tree_requests_that_end_behind_one_another(fmt, n, H, per_range):
    """Ranges whose last tile is a whole request right behind another request's end, with sums that differ by orders
    of magnitude: each request is divided by its own sum, in every call."""
    rng = np.random.default_rng(per_range)
    blocks = -(-n * H // 128)
    B = 76 // blocks * per_range                        # one tile each
    lens = np.where(np.arange(B) % 2, rng.integers(n, n + 4, B), rng.integers(230, 257, B)).astype(np.int32)
    t = Tree(per_range, lens, n, H, fmt=fmt, bs=64)
    out, lse = t.run()
    t.check((out, lse))
    for _ in range(20):
        again = t.run()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def rounds_by_much():
    """x on bf16's grid whose exp(-x) rounds to bf16 up and down by most of half a step."""
    x = O.bf16_to_f64(np.arange(0x3f00, 0x4080, dtype=np.uint16))          # 0.5 .. 4
    p = np.exp(-x)
    by = O.bf16_to_f64(O._f32_to_bf16_bits(p.astype(np.float32))) / p - 1
    return float(x[by.argmax()]), float(x[by.argmin()])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(1, 16), (2, 16), (4, 16), (5, 16), (8, 32)])
def test_tree_weights_that_round_alike(fmt, n, H):
    """One key with weight 1 and 199 whose weights round to bf16 the same way, by nearly half a step: where all rows
    are the same the result is that row whatever the weights, so what a weight's rounding adds to the sum of products
    has to be in the sum it is divided by.  (Divided by the unrounded weights' sum it would be off by 2^-8 of itself,
    a whole step of bf16 below 2.)  The log-sum-exp is of the weights as they are: 200 additions, the 2-ulp
    exponential and logarithm, 300 u relative to the sum."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    value = 255 / 128                                   # all mantissa bits: steps are 2^-8 of it
    for x in rounds_by_much():
        rows = np.zeros((256, 576))
        rows[:, :512] = value
        rows[1:, 512] = -x
        kv = O._f32_to_bf16_bits(rows.astype(np.float32))
        cache = bf(kv) if fmt == "bf16" else torch.from_numpy(O.kv_fp8_quantize(kv, 64)).cuda()
        q = torch.zeros(1, n, H, 576, dtype=BF, device="cuda")
        q[..., 512] = 1
        mask = torch.full((1, n), (1 << n) - 1, device="cuda")
        out, lse = dsa.dsa_tree_decode(q, cache, i32([list(range(4))]), i32([200]), mask, 64, 1.0)
        assert torch.equal(out, torch.full_like(out, value)), (out.float().min(), out.float().max())
        want = np.log(1 + 199 * np.exp(-x))
        assert np.abs(f64(lse) - want).max() <= 300 * U + 4 * U * want
        assert bad_count() == 0


@pytest.mark.parametrize("n,H", [(2, 16), (3, 16)])
def test_tree_last_positions_of_31_bits(n, H):
    """A request that fills a table of 2^31 - 1 positions and more: its drafted tokens, in the last tile, are seen."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    bs = 1 << 16
    blocks = (1 << 31) // bs
    rng = np.random.default_rng(n)
    rows = np.zeros((2 * bs, 576), dtype=np.float32)    # (the context's scores are 0)
    last = (1 << 31) - 1 - n                            # first drafted position
    at = bs + last % bs                                 # its row: the last block is the second of the cache's
    drafted = rng.standard_normal((n, 576)).astype(np.float32)
    drafted[:, 512] = 60                                # (a score of 60 outweighs 2^31 of 0 by e^38)
    rows[at:at + n] = drafted
    kv = O._f32_to_bf16_bits(rows)
    bt = np.zeros((1, blocks), dtype=np.int32)
    bt[0, -1] = 1
    q = torch.zeros(1, n, H, 576, dtype=BF, device="cuda")
    q[..., 512] = 1
    mask = [1 << i for i in range(n)]                   # each sees itself alone
    out, lse = dsa.dsa_tree_decode(q, bf(kv), i32(bt), i32([(1 << 31) - 1]), torch.from_numpy(signed([mask])).cuda(), bs, 1.0)
    assert bad_count() == 0
    want = O.bf16_to_f64(kv[at:at + n, :512])[None, :, None]
    assert np.abs(f32(out) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-12
    assert np.abs(f64(lse) - 60).max() <= 60 * 8 * U


@pytest.mark.parametrize("as_handle", [False, True])
def test_gradient_of_a_side_without_heads_on_another_stream(as_handle):
    """The weights' gradient of a side without heads is zeros, there in the order of the call's stream and that
    stream's memory: not a block that the current stream's queued kernels still write."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    c = Norm(3, 40, 4, 2, 192)
    c.x[0], c.g[0] = c.x[0][:, :0], c.g[0][:, :0]
    want = c.gradient()
    torch.cuda.synchronize()
    pos = i32(c.pos)
    s = torch.cuda.Stream()
    for i in range(3):
        with torch.cuda.stream(s):                      # (blocks of that stream that hold something else)
            old = [torch.full((192,), 5.0, device="cuda") for _ in range(8)]
        spare = [torch.full((192,), 3.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        blocks = {x.data_ptr() for x in spare}
        torch.cuda._sleep(20_000_000)
        for x in spare:
            x.fill_(1)
        del spare, x, old
        got = dsa.dsa_qk_norm_rope_gradient(*c.g, *c.x, *c.w, pos, c.freqs, eps=c.eps, stream=s.cuda_stream if as_handle else s)
        with torch.cuda.stream(s):
            seen = got[2].clone()
        s.synchronize()                                 # (the current stream still sleeps)
        assert not torch.cuda.current_stream().query()
        with torch.cuda.stream(s):
            assert seen.tolist() == [0.0] * 192 and got[2].data_ptr() not in blocks
        torch.cuda.synchronize()
        assert torch.equal(got[3], want[3]) and (got[2] == 0).all()


FIRST_USE = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import os
import subprocess
import sys

import numpy as np
import torch
import dsa_sparse_mla_prefill_gb300 as dsa
import oracle.dsa_oracle as O
from gpu_util import bf, i32
from test_gpu_draft_step import Norm, Tree, bad_count
sizes = [(4, 16, 'bf16'), (2, 16, 'bf16'), (8, 16, 'fp8'), (3, 16, 'fp8')]
trees = [Tree(i, [900, 33, 600], n, H, fmt=fmt, bs=64) for i, (n, H, fmt) in enumerate(sizes) for _ in range(2)]
norms = [Norm(9, 50, 4, 2, 192), Norm(9, 50, 4, 2, 192)]
moved = torch.arange(64 * 576, device='cuda').reshape(64, 576).to(torch.bfloat16)
before, table, lens, keep = moved.clone(), i32([[0]]), i32([9]), i32([[1, 3, -1, -1]])
work = [t.run for t in trees] + [c.forward for c in norms] + [c.gradient for c in norms]
work.append(lambda: dsa.dsa_kv_keep(moved, table, lens, keep, 64, 4))
start, got, streams = threading.Barrier(len(work)), [None] * len(work), [torch.cuda.Stream() for _ in work]
torch.cuda.synchronize()

def one(i):
    with torch.cuda.stream(streams[i]):
        start.wait()
        try:
            got[i] = work[i]()
        except Exception as e:
            got[i] = e
threads = [threading.Thread(target=one, args=(i,)) for i in range(len(work))]
for x in threads: x.start()
for x in threads: x.join()
torch.cuda.synchronize()
wrong = [(i, g) for i, g in enumerate(got) if isinstance(g, Exception)]
assert not wrong, wrong
for t, g in zip(trees, got): t.check(g)
for c, g in zip(norms, got[8:10]): c.check_forward(g)
for c, g in zip(norms, got[10:12]): c.check_gradient(g)
before[[5, 6]] = before[[6, 8]]
assert got[12].tolist() == [7] and torch.equal(moved, before) and bad_count() == 0
print('all right')
"""


def test_first_calls_of_a_process_from_several_threads():
    """Every operator's first call at the same time as the others', two of each kernel: what a call keeps for later
    ones (the devices, attributes, the tensor maps' encoder) is complete for whoever uses it."""
    here = os.path.dirname(os.path.abspath(__file__))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", FIRST_USE.format(root=os.path.dirname(here), tests=here)], capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip().endswith("all right"), r.stderr[-2000:]


@pytest.mark.parametrize("T,Hq,Hk,d,d_norm", [(100003, 1, 0, 128, None), (20001, 5, 3, 64, None), (25001, 4, 1, 256, None),
                                              (100001, 1, 0, 576, 512), (20001, 5, 2, 70, None)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradient_counts_every_row_once(T, Hq, Hk, d, d_norm, dtype):
    """Inputs and gradients of 1 and -1, weights of 1: a row's r is 1 within 4 u and its terms are 1 or -1, so a row
    left out or added twice changes every column's sum by one.  The sums are integers; a lane adds the rows of its
    share of at least 152 x 8 workers one after another, its warp's lanes, its CTA's warps and the CTAs' partial sums
    (38 and 8 in a column) are less than 60 additions more: (rows / 1216 + 64) u of the number of rows, which is below
    one."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(d)

    def signs(H):
        t = torch.from_numpy(rng.integers(0, 2, (T, H, d), dtype=np.int8)).cuda()
        return (t * 2 - 1).to(dtype)
    n = d_norm or d
    one = torch.ones(n, dtype=dtype, device="cuda")
    x = [signs(H) if H else None for H in (Hq, Hk)]
    g = [signs(H) if H else None for H in (Hq, Hk)]
    got = dsa.dsa_qk_norm_rope_gradient(*g, *x, one, one if Hk else None, None, None, eps=0.0, d_norm=d_norm)
    for a, b, w in zip(x, g, got[2:]):
        if a is None:
            assert w is None
            continue
        want = (a[..., :n] * b[..., :n]).double().sum((0, 1))
        rows = a.shape[0] * a.shape[1]
        tol = (rows / 1216 + 64) * U * rows
        assert tol < 1
        assert (w.double() - want).abs().max().item() <= tol


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(2, 16), (5, 16), (4, 64)])
def test_tree_chain_is_the_decode_steps(fmt, n, H):
    """A chain of drafted tokens attended at once is what attending them one after another gives: both within the
    decode step's bound (test_gpu_decode_step.py) of the same exact result, element by element, so within two of it of
    each other."""
    import dsa_sparse_mla_prefill_gb300 as dsa
    t = Tree(n, [300, 1029, 64, 4000], n, H, fmt=fmt, bs=64, mask=[ancestors(range(-1, n - 1))] * 4)
    got = t.run()
    t.check(got)
    q, cache, bt, lens, _, bs, scale = t.args()
    tiles = -(-int(t.lens.max()) // 128)
    for i in range(n):
        out, lse = dsa.dsa_paged_decode(q[:, i].contiguous(), cache, bt, lens - (n - 1 - i), bs, scale)
        ref = O.paged_decode(t.q[:, i], t.values, t.bt, t.lens - (n - 1 - i), bs, scale)
        score = 1155 * U * ref["mass"]
        tol = (2 * (2.0 ** -8 + score) * (1 + 2.0 ** -7))[..., None] * ref["spread"] + 2.0 ** -8 * np.abs(ref["out"]) + 1e-30
        ltol = score + 2.0 ** -21 + (tiles + 32) * U + 4 * U * np.abs(ref["lse"])
        assert (np.abs(f32(out) - ref["out"]) <= tol).all() and (np.abs(f64(lse) - ref["lse"]) <= ltol).all()
        assert (np.abs(f32(got[0][:, i]) - f32(out)) <= 2 * tol).all() and (np.abs(f64(got[1][:, i]) - f64(lse)) <= 2 * ltol).all()
    assert bad_count() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(2, 16), (8, 16), (8, 32)])
def test_tree_one_long_request_among_short_ones(fmt, n, H):
    """A request that most of the ranges share while the batch's average is a few: its many parts are joined whatever
    the join was launched for."""
    lens = [300] * 31
    lens.insert(11, 40000)
    t = Tree(n, lens, n, H, fmt=fmt, bs=64)
    t.check(t.run())
