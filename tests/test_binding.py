"""What the Python binding refuses before anything reaches the library (no GPU)."""
import pytest

import dsa_sparse_mla_prefill_gb300 as dsa


def test_no_stream_of_a_host_tensor():
    """A call takes its stream from a tensor's device: host tensors, which the strided call is not asked about
    otherwise, are refused there and never reach a kernel as addresses."""
    import torch
    with pytest.raises(ValueError):
        dsa._stream(None, torch.device("cpu"))
    q, k, v = (torch.zeros(4, 2, 256, dtype=torch.bfloat16) for _ in range(3))
    with pytest.raises(ValueError):
        dsa.dsa_masked_mha_prefill_strided(q, k, v, torch.zeros(4, 4, dtype=torch.int32), 1.0)


def test_a_frequency_table_is_its_callers_own():
    from dsa_sparse_mla_prefill_gb300 import build as b
    b.build()
    mine = dsa.dsa_rope_freqs(64, mscale=1.25)
    turns = list(mine.turns)
    mine.mscale, mine.turns[3], mine.layout = 7.0, 0, 1
    other = dsa.dsa_rope_freqs(64, mscale=1.25)
    assert (other.mscale, other.layout, list(other.turns)) == (1.25, 0, turns)
