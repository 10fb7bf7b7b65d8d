"""Refusals of the AdamW entry point's flags (nothing is launched, so no GPU is
needed)."""
import ctypes

from multiresolution_hash_grid_amd import hashgrid as B
from multiresolution_hash_grid_amd import residual as R


def test_clearing_skipped_gradients_alone_is_refused():
    # HG_ADAM_ZERO_SKIPPED says when HG_ADAM_ZERO_GRAD clears; without it there is nothing to say.
    lib, o = R._lib(), R._AdamW(0.9, 0.99, 1e-8, 1, 0)
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 0, None, R.HG_ADAM_ZERO_SKIPPED, None) == B.HG_EINVAL
    assert "HG_ADAM_ZERO_GRAD" in lib.hashgrid_last_error().decode()
    both = B.HG_ADAM_ZERO_GRAD | R.HG_ADAM_ZERO_SKIPPED
    assert lib.hashgrid_adamw_step(ctypes.byref(o), None, 0, None, both, None) == B.HG_OK
