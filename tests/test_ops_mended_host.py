"""What moe_rope and its tables refuse beside what tests/test_more_ops_host.py has, and what the binding hands to the library; no
GPU is needed.  The handle and the pointers here are never followed."""
import pytest

import bit_moe_decode_02_gb300 as moe
from test_more_ops_host import A, INV, L, o, rope  # noqa: F401


@pytest.mark.parametrize("kw,word", [
    (dict(position=9 * A), "q_out overlaps position"), (dict(position=9 * A - 8), "q_out overlaps position"),
    (dict(position=9 * A + 512 * 2 * 3 - 4), "q_out overlaps position"), (dict(turns=9 * A + 1024), "q_out overlaps turns"),
    (dict(turns=10 * A - 248), "k_out overlaps turns"), (dict(position=10 * A + 4), "k_out overlaps position"),
    (dict(qos=520, position=9 * A + 1032), "q_out overlaps position"),                                # from the gap into the next row
    (dict(q=9 * A, qs=512, position=9 * A + 512), "q_out overlaps position"),                         # in place
    (dict(qos=512 + 128, turns=9 * A + 1280 + 1024 + 8), "q_out overlaps turns")])
def test_rope_outputs_over_positions_or_the_table(L, o, kw, word):  # noqa: F811
    """Another token's row would overwrite a position or a speed before it is read."""
    assert rope(L, o, **kw) == INV and word in moe.moe_last_error()


def test_rope_positions_beside_the_outputs(L, o):  # noqa: F811
    """What ends where an output begins, begins where it ends, or lies between two of its rows is no overlap: the check after it,
    of the outputs' own, is what refuses these."""
    for kw in (dict(position=9 * A - 12), dict(position=9 * A + 512 * 2 * 3), dict(turns=9 * A - 256), dict(qos=520, position=9 * A + 1024),
               dict(qos=512 + 128, turns=9 * A + 1024), dict(qos=512 + 128, turns=9 * A + 1280 + 1024)):
        assert rope(L, o, ko=9 * A + 16, kos=kw.get("qos", 512), **kw) == INV and "q_out overlaps k_out" in moe.moe_last_error()
