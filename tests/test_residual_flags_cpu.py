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


def test_counted_steps_need_their_counts():
    lib = R._lib()
    t = (R._AdamWTensor * 1)(R._AdamWTensor(param=0x1000, grad=0x1000, m=0x1000, v=0x1000, count=0, lr=1e-3, state_bits=32))
    o = R._AdamW(0.9, 0.99, 1e-8, 0, 0, None)  # the step's number is not looked at
    assert lib.hashgrid_adamw_step(ctypes.byref(o), t, 1, None, R.HG_ADAM_CLOCK, None) == B.HG_EINVAL
    assert "clocks" in lib.hashgrid_last_error().decode()
    o = R._AdamW(0.9, 0.99, 1e-8, 0, 0, 0x1002)
    assert lib.hashgrid_adamw_step(ctypes.byref(o), t, 1, None, R.HG_ADAM_CLOCK, None) == B.HG_EINVAL
    o = R._AdamW(0.9, 0.99, 1e-8, 0, 0, 0x1000)
    assert lib.hashgrid_adamw_step(ctypes.byref(o), t, 1, None, R.HG_ADAM_CLOCK, None) == B.HG_OK
    assert lib.hashgrid_adamw_step(ctypes.byref(o), t, 1, None, 0, None) == B.HG_EINVAL
    assert "step" in lib.hashgrid_last_error().decode()
