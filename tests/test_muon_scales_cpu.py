"""Refusals of coefficients whose update would leave the range of the tiled products' 16-bit parts (CPU only: nothing is
launched)."""
import pytest

from kronecker_factored_structured_amd import _lib
from test_finetune_cpu import MB, P, muon

BIG = ((P(), P(MB), P(2 * MB), 1, 128, 128),)      # does not fit LDS
STEEP = dict(a=8.28721201814563, b=-23.595886519098837, c=17.300387312530933)


@pytest.mark.parametrize("kw", [dict(STEEP, steps=5), dict(a=1025.0, b=0.0, c=0.0, steps=1), dict(a=2.0, b=0.0, c=0.0, steps=12),
                                dict(a=1e38, b=1e38, c=1e38, steps=16), dict(a=0.0, b=0.0, c=-1e5, steps=2), dict(a=0.0, b=2000.0, c=0.0, steps=1)])
def test_growth_is_refused(kw):
    assert muon(tensors=BIG, **kw) == _lib.KRON_E_UNSUPPORTED, _lib.last_error()
    assert "singular value" in _lib.last_error()
    # (what is wrong whatever the coefficients are comes first)
    assert muon(tensors=BIG, ws=None, **kw) == _lib.KRON_E_WORKSPACE


def test_workspace_of_many_large_matrices():
    """Matrices of one size share a workspace: it grows with their number up to where a few fill the GPU."""
    import ctypes

    def ws(count, rows, cols, dtype):
        return _lib.lib().kron_muon_workspace_bytes(1, (ctypes.c_int64 * 1)(count), (ctypes.c_int32 * 1)(rows), (ctypes.c_int32 * 1)(cols), dtype)

    for dtype, most in ((0, 4.6e9), (1, 2.3e9)):
        for side, enough in ((4096, 16), (16384, 1), (5000, 10)):
            assert 0 < ws(1, side, side, dtype) <= ws(64, side, side, dtype) == ws(enough, side, side, dtype) == ws(1 << 20, side, side, dtype) < most
        assert ws(64, 1024, 1024, dtype) == 64 * ws(1, 1024, 1024, dtype) == ws(65, 1024, 1024, dtype)
        assert ws(7, 65, 16384, dtype) == pytest.approx(7 * ws(1, 65, 16384, dtype), rel=1e-3)
