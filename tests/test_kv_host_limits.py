"""K/V cache entry points without a GPU: arguments at the ends of their ranges."""
import pytest

from block_sparse_attention_select_gb300 import build as qbuild
from block_sparse_attention_select_gb300 import qsa
from test_kv_host import _attend


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qsa.load()


def test_scale_times_log2_e_must_be_finite(lib):
    for scale in (2.4e38, 3.4e38):
        assert _attend(lib, scale=scale) == qsa.QSA_ERR_INVALID_ARG
    for scale in (1e-38, 2.3e38):
        assert _attend(lib, scale=scale) == qsa.QSA_ERR_NO_DEVICE
