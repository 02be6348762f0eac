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
