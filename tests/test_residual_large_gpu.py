"""Steps and gradients of more than 2^32 threads in one launch."""
import pytest
import torch

import multiresolution_hash_grid_amd as hg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_adamw_over_more_values_than_a_grid_dimension_has_threads():
    # Two tensors of 2^33 values and some: 2^32 threads and some at 4 values each.  8-bit moments, 16-bit gradients: 128 GiB.
    counts = [(1 << 33) + 5, (1 << 33) + 700]
    if torch.cuda.get_device_properties(0).total_memory < 160 << 30:
        pytest.skip("needs 160 GiB of device memory")
    tensors = []
    for n in counts:
        p = torch.ones(n, device=DEV)
        tensors.append(hg.AdamWTensor(param=p, grad=torch.ones(n, device=DEV, dtype=torch.bfloat16), lr=0.25,
                                      **hg.AdamWTensor.states(p, 8)))
    hg.hashgrid_adamw_step(tensors, step=1, eps=0.0)
    for t in tensors:
        # the first step of a constant gradient is lr
        low, high = t.param.aminmax()
        assert abs(float(low) - 0.75) <= 1e-6 and abs(float(high) - 0.75) <= 1e-6
        # exponents: m = 0.1 in [2^-4, 2^-3), v = 0.001 in [2^-10, 2^-9)
        assert t.m_exp.aminmax() == (127 - 4 - 7,) * 2 and t.v_exp.aminmax() == (127 - 10 - 15,) * 2
    del tensors, t, p
    torch.cuda.empty_cache()


def test_gradients_of_a_very_large_weight_without_rows():
    n, k = 65536, 8192
    w = torch.empty(n, k, dtype=torch.float16, device=DEV)
    dw, db = torch.ones(n, k, dtype=torch.float16, device=DEV), torch.ones(n, device=DEV)
    e = torch.empty(0, k, dtype=torch.float16, device=DEV)
    dy = torch.empty(0, n, dtype=torch.float16, device=DEV)
    hg.hashgrid_linear_backward(dy, e, w, dw=dw, db=db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    hg.hashgrid_linear_backward(dy, e, w, dw=dw, db=db)
    assert not dw.any() and not db.any()
