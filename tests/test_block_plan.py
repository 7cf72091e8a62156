"""How the norm backward deals its rows, read from the workspace it asks for.
No GPU needed."""
import pytest

import deterministic_attention_gb300 as da


@pytest.fixture(scope="module")
def L():
    da.build()
    return da.lib()


def _up(x):
    return (x + 255) // 256 * 256


@pytest.mark.parametrize("d", [64, 768, 4096])
@pytest.mark.parametrize("rows,G", [(10, 100), (8, 250), (7, 90), (100, 3), (5, 2), (1000, 7), (11, 55),
                                    (3, 200), (1024, 32), (2, 304), (9, 303), (1 << 14, 2)])
def test_no_slice_of_a_gate_row_is_empty(L, rows, G, d):
    """Each of the G gate rows shared by `rows` rows is cut into equal slices
    (the last may be shorter): about four for each of 152 blocks, and every one
    with a row in it."""
    want = max(1, min(4 * 152 // G, rows))
    per = -(-rows // want)
    slices = -(-rows // per)
    assert (slices - 1) * per < rows
    blocks = min(G * slices, 152)
    expect = 2 * _up(blocks * d * 4) + (_up(G * slices * d * 4) if slices > 1 else 0)
    assert L.block_norm_bwd_workspace_bytes(rows * G, d, G) == expect
