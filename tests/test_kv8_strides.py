"""Row strides of dimensions with a single entry, which programs and exchange
formats fill in as they like: not looked at (host validation, no GPU, dummy
pointers)."""
import pytest
import torch

from gated_block_sparse_token_b200 import build as B
from gated_block_sparse_token_b200 import sas

from test_kv8_abi import FAKE, INVALID, cfg, kv8, rows

nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host validation runs on CPU-only hosts")


@pytest.fixture(scope="module")
def L():
    B.build()
    return sas.lib()


@nogpu
def test_single_entries_have_any_stride(L):
    """Past the validation a call fails for want of a GPU, which is another status."""
    odd = [dict(seq_stride=1), dict(seq_stride=-3), dict(token_stride=1, tokens=1), dict(token_stride=-8, tokens=1)]
    one = cfg(num_q_heads=1, num_kv_heads=1)
    for o in odd + [dict(head_stride=7)]:
        t = o.get("tokens", 64)
        r = rows(**o)
        assert L.sas_qk_norm_rope(one, r, r, FAKE, FAKE, None, 1, t, 1e6, r, r, None) == sas.SAS_ERR_CUDA, o
        assert L.sas_kv8_append(one, kv8(batch=1), r, r, None, None, 1, FAKE, 256, None) == sas.SAS_ERR_CUDA, o
        assert L.sas_kv8_read(one, kv8(batch=1), None, t, r, r, FAKE, 256, None) == sas.SAS_ERR_CUDA, o
    two = cfg(num_q_heads=2, num_kv_heads=2)
    for o in (dict(seq_stride=1), dict(head_stride=7), dict(token_stride=1), dict(seq_stride=-8), dict(token_stride=-128)):
        r = rows(**o)
        assert L.sas_qk_norm_rope(two, r, r, FAKE, FAKE, None, 2, 64, 1e6, r, r, None) == INVALID, o
        assert L.sas_kv8_append(two, kv8(), r, r, None, None, 1, FAKE, 256, None) == INVALID, o
        assert L.sas_kv8_read(two, kv8(), None, 64, r, r, FAKE, 256, None) == INVALID, o
    assert L.sas_kv8_append(one, kv8(batch=1), rows(tokens=-1), rows(), None, None, 1, FAKE, 256, None) == INVALID
