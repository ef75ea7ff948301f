"""Arguments of rotary_table and of the calls that make tensors, on a machine without a GPU."""
import pytest
import torch

from block_sparse_attention_select_gb300 import qsa
from test_block_layer_host import BAD, GO, _table, lib  # noqa: F401


def test_amplitudes_past_fp32_are_refused(lib):  # noqa: F811
    """The table holds FP32 numbers: an amplitude past them would fill it with infinities
    (and NaN, where they meet a sine of zero)."""
    for a in (3.5e38, 1e300):
        for kind in (1, 2, 3):
            assert _table(lib, kind, amplitude=a) == BAD
    assert _table(lib, 1, amplitude=3.4e38) == GO and _table(lib, 3, amplitude=1e-30) == GO


@pytest.mark.parametrize("device,want", [(0, 0), (1, 1), ("cuda:0", "cuda:0"), (torch.device("cuda", 0), torch.device("cuda", 0)),
                                         (None, "cuda")])
def test_device_number_0_is_that_device(monkeypatch, device, want):
    """Not the current one, which another device may be."""
    asked = []

    class Asked(Exception):
        pass

    def empty(*a, **kw):
        asked.append(kw["device"])
        raise Asked

    monkeypatch.setattr(qsa.torch, "empty", empty)
    for call in (lambda: qsa.Batch.empty(2, 3, device), lambda: qsa.rotary_table(4, 16, device=device),
                 lambda: qsa.rope_table(4, 16, device=device), lambda: qsa.alloc_workspace(4, 16, 2, device)):
        with pytest.raises(Asked):
            call()
    assert asked == [want] * 4
