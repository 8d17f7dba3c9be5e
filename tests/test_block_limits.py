"""Sizes at the end of the range of the sorted tokens' calls: refused before any arithmetic on them leaves 64 bits (no GPU needed)."""
import ctypes

import pytest

from routed_expert_ffn_layer_amd import moe

MANY, FAR = (1 << 31) - 1, 1 << 36


def _p(mb):
    return ctypes.c_void_p(mb << 20)


@pytest.mark.parametrize("n_rows,ld", [(MANY, FAR), (MANY, 1 << 29), ((1 << 24) + 1, 1 << 35)])
def test_rows_beyond_any_memory(n_rows, ld):
    """The size in bytes of so many rows passes 2^64, and the overlap with the other buffers went unseen."""
    L = moe.lib()
    for what, call in (
            ("rows", lambda: L.moe_dispatch(_p(64), 1, 64, _p(1), 4, 2, 8, 64, _p(2), _p(3), _p(4), _p(5), _p(16), ld, n_rows, None, 0, None)),
            ("rows", lambda: L.moe_combine_rows(_p(16), 1, ld, n_rows, _p(1), _p(2), 4, 2, 64, _p(17), 1, 64, None)),
            ("rows", lambda: L.moe_dispatch_backward(_p(16), 1, ld, n_rows, _p(2), 4, 2, 64, _p(17), 1, 64, None)),
            ("rows", lambda: L.moe_combine_rows_backward(_p(15), 1, 64, _p(16), 1, ld, n_rows, _p(1), _p(2), 4, 2, 64, _p(17), 64, _p(3), None)),
            ("d_rows", lambda: L.moe_combine_rows_backward(_p(15), 1, 64, _p(17), 1, 64, n_rows, _p(1), _p(2), 4, 2, 64, _p(16), ld, _p(3), None))):
        assert call() == moe.MOE_EINVAL
        assert L.moe_last_error().decode().startswith(what + ": ") and "in all" in L.moe_last_error().decode()
