"""Calls on a stream that is not the current one: the tensors that the binding makes for them."""
import numpy as np
import pytest

from gpu_util import bf, i32, need_gpu, torch
from synth import normal_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def decode_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(1)
    cache, q = bf(normal_bf16(rng, (4096, 576))), bf(normal_bf16(rng, (3, 32, 576)))
    table, lens = i32(rng.permutation(64).reshape(1, 64).repeat(3, 0)), i32([4000, 77, 1500])
    return lambda **kw: dsa.dsa_paged_decode(q, cache, table, lens, 64, 192 ** -0.5, **kw)


def rope_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    x, pos = bf(normal_bf16(np.random.default_rng(2), (700, 16, 64))), i32(np.arange(700))
    freqs = dsa.dsa_rope_freqs(64)
    return lambda **kw: (dsa.dsa_rope(x, pos, freqs, **kw),)


def prefill_inputs():
    rng = np.random.default_rng(3)
    q, kv = bf(normal_bf16(rng, (300, 16, 576))), bf(normal_bf16(rng, (2000, 576)))
    return q, kv, i32(np.sort(rng.integers(0, 300, (300, 128)), axis=1) % (1 + np.arange(300))[:, None])


def sparse_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    q, kv, idx = prefill_inputs()
    return lambda **kw: dsa.dsa_sparse_prefill(q, kv, idx, 128, 0.07, **kw)


def sparse_fp8_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    q, kv, idx = prefill_inputs()
    rows = dsa.dsa_kv_fp8_quantize(kv, 64)
    return lambda **kw: dsa.dsa_sparse_prefill_fp8(q, rows, idx, 128, 0.07, **kw)


def union_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    idx = prefill_inputs()[2]

    return lambda **kw: dsa.dsa_union_build(idx, 128, 8, 2000, **kw)


def grouped_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    q, kv, idx = prefill_inputs()
    u, n, m = dsa.dsa_union_build(idx, 128, 8, 2000)
    return lambda **kw: dsa.dsa_grouped_prefill(q, kv, u, n, m, 8, 0.07, **kw)


def key_mask_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    idx = prefill_inputs()[2]
    return lambda **kw: (dsa.dsa_topk_to_key_mask(idx, 128, 64, **kw),)


def convert_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    idx, table = prefill_inputs()[2], i32(np.arange(40)[None, ::-1].copy())
    return lambda **kw: (dsa.dsa_local_to_global(idx, 128, [2000], table, 50, 2000, **kw),)


def masked_inputs():
    import dsa_sparse_mla_prefill_gb300 as dsa
    rng = np.random.default_rng(4)
    q, k, v = (bf(normal_bf16(rng, (300, 4, 256))) for _ in range(3))
    return q, k, v, dsa.dsa_topk_to_key_mask(prefill_inputs()[2], 128, 12)


def masked_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    a = masked_inputs()
    return lambda **kw: dsa.dsa_masked_mha_prefill(*a, 0.06, **kw)


def masked_strided_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    a = masked_inputs()
    return lambda **kw: dsa.dsa_masked_mha_prefill_strided(*a, 0.06, **kw)


def quantize_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    kv = prefill_inputs()[1]
    return lambda **kw: (dsa.dsa_kv_fp8_quantize(kv, 64, **kw),)


def dequantize_call():
    import dsa_sparse_mla_prefill_gb300 as dsa
    rows = dsa.dsa_kv_fp8_quantize(prefill_inputs()[1], 64)
    return lambda **kw: (dsa.dsa_kv_fp8_dequantize(rows, 64, **kw),)


CALLS = {"decode": decode_call, "rope": rope_call, "sparse": sparse_call, "sparse_fp8": sparse_fp8_call,
         "union": union_call, "grouped": grouped_call, "key_mask": key_mask_call, "convert": convert_call,
         "masked": masked_call, "masked_strided": masked_strided_call, "quantize": quantize_call,
         "dequantize": dequantize_call}


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_results_are_not_memory_that_the_current_stream_still_uses(name, as_handle):
    """Blocks of the results' sizes, freed on the current stream behind a kernel that will yet write them: a call on
    another stream, which waits for nothing, gets none of them, and neither does any harm to the other."""
    call = CALLS[name]()
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    import dsa_sparse_mla_prefill_gb300 as dsa
    spare = [torch.empty_like(t) for t in want for _ in range(2)] + \
        [torch.empty(dsa.dsa_paged_decode_workspace(3, 32, 4096), dtype=torch.uint8, device="cuda")]
    torch.cuda.synchronize()
    blocks = {t.data_ptr() for t in spare}
    torch.cuda._sleep(20_000_000)
    for t in spare:
        t.fill_(1)
    del spare, t
    got = call(stream=s.cuda_stream if as_handle else s)
    assert not blocks & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", list(CALLS))
def test_the_default_stream_by_its_handle(name):
    """Handle 0 from inside another stream: the default stream, not the current one."""
    call = CALLS[name]()
    want = call()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(stream=0)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["decode", "rope", "sparse"])
def test_calls_on_a_side_stream_of_a_capture(name):
    """A captured step that forks to another stream and joins again, replayed with other kernels in between."""
    call = CALLS[name]()
    want = call()
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        first = call(stream=s)
        second = call(stream=s)
        here.wait_stream(s)
        third = call()
    for _ in range(3):
        for t in first + second + third:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        for got in (first, second, third):
            for a, b in zip(got, want):
                assert torch.equal(a, b)
