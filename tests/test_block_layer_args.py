"""Arguments of rotary_table and of the calls that make tensors, on a machine without a GPU."""
from test_block_layer_host import BAD, GO, _table, lib  # noqa: F401


def test_amplitudes_past_fp32_are_refused(lib):  # noqa: F811
    """The table holds FP32 numbers: an amplitude past them would fill it with infinities
    (and NaN, where they meet a sine of zero)."""
    for a in (3.5e38, 1e300):
        for kind in (1, 2, 3):
            assert _table(lib, kind, amplitude=a) == BAD
    assert _table(lib, 1, amplitude=3.4e38) == GO and _table(lib, 3, amplitude=1e-30) == GO
