"""GPU: what the E4M3 cache's codes stand for, each of them at each scale byte."""
import numpy as np
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from oracle import kv_cache as O

pytestmark = pytest.mark.gpu


def test_every_code_at_every_scale_byte_reads_back():
    """256 scale bytes x 256 codes: code * 2^(byte - 127) with the byte held to
    112 .. 135; the seven codes above 240 (256, 288, ..
    448) at 2^8 are past FP16 and read as infinity."""
    D, page = 256, 64
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").expand(4, page, 1, D).contiguous()
    scale = torch.arange(256, dtype=torch.uint8, device="cuda").view(4, page, 1).contiguous()
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None].contiguous()
    f8 = codes.view(torch.float8_e4m3fn)
    cache = qsa.KVCache(f8, f8.clone(), table, scale, scale.clone())
    got = qsa.kv_load(torch.tensor([0, 256], dtype=torch.int32, device="cuda"),
                      torch.tensor([0], dtype=torch.int32, device="cuda"), 256, cache)
    assert qsa.get_device_status() == qsa.QSA_OK
    byte = np.clip(np.arange(256), 112, 135)
    with np.errstate(over="ignore"):
        want = (O.e4m3_values()[None] * 2.0 ** (byte - 127.0)[:, None]).astype(np.float16)
    assert np.isinf(want).sum() == 2 * 7 * (256 - 135)
    for x in got:
        np.testing.assert_array_equal(x.cpu().numpy()[:, 0], want)
