"""The 8-bit cache's write, read-back and attention at the ends of their ranges
and in the loops that only many blocks reach.

Attention over few distinct pages that many blocks share: the float64 side then
weighs every page by how often it is listed."""
import pytest
import torch

from gated_block_sparse_token_b200 import sas

import kv8_testlib as K

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = [K.E4M3, K.INT8]
INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1


def status(ws):
    torch.cuda.synchronize()
    return sas.get_device_status(ws)


def test_append_lengths_at_the_ends_of_int32():
    """A length that no count can be taken from is reported like every other bad one, and writes nothing."""
    lens = [INT_MIN, INT_MIN + 3, -1, INT_MAX, 70]
    cfg = sas.Config(1, 1)
    kv = K.make_cache(5, 1, 4, K.INT8, False, [70] * 5, DEV, seed=2)
    x = torch.randn((5, 1, 70, 128), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    before = [t.clone() for t in (kv.k.view(torch.uint8), kv.v.view(torch.uint8), kv.k_scale, kv.k_tail.view(torch.int16),
                                  kv.v_tail.view(torch.int16))]
    new = torch.tensor([1, 70, 70, 70, 70], dtype=torch.int32, device=DEV)
    for n in (None, new):
        ws = sas.make_workspace(cfg, DEV)
        kv.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        sas.kv8_append(cfg, kv, x, x, ws, new_lens=n)
        assert status(ws) == sas.SAS_ERR_DEVICE_BOUNDS
        for t, b in zip((kv.k.view(torch.uint8), kv.v.view(torch.uint8), kv.k_scale, kv.k_tail.view(torch.int16),
                         kv.v_tail.view(torch.int16)), before):
            assert torch.equal(t[:4], b[:4])
        assert torch.equal(kv.k_tail[4, 0, :6].cpu(), x[4, 0, 64:].cpu())
