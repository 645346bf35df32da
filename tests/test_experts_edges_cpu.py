"""The routed-FFN entry points on the host at the edges of their types and sizes
(no GPU needed)."""
import numpy as np
import pytest

from oracle import experts_oracle as O

P = pytest.importorskip("free_ffn_activation_amd.prox",
                        reason="libprox.so not built (run __graft_entry__.build())")


def test_oracle_holds_quotients_at_the_largest_code():
    """642 steps of 2^-149: the scale is one step, a quotient of 642 has no code."""
    x = np.zeros((1, 128), np.float32)
    x[0, :4] = np.array([642, -642, 214, 1]) * 2.0 ** -149
    q, s = O.quantize(x, 1)
    assert s[0, 0] == np.float32(2.0 ** -149)
    assert q[0, :4].tolist() == [448, -448, 208, 1]
