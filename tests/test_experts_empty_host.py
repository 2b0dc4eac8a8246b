"""Refusals of the weight gradient of no tokens, before any CUDA work (CPU only)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def qb():
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


def test_weight_gradient_of_no_columns(qb):
    F, ODD, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None
    # one group: empty operands have no address, and what is added to stays
    ok = [NUL, NUL, NUL, NUL, NUL, 1, 0, 64, 48, F, 0, 1, NUL]
    assert qb.lib.qb_fp8_expert_wgrad(*ok) == qb.QB_OK
    for i, v, want in [(0, ODD, qb.QB_EINVAL), (3, ODD, qb.QB_EINVAL), (5, 0, qb.QB_EINVAL),
                       (6, -128, qb.QB_EINVAL), (6, 128, qb.QB_EINVAL), (7, 0, qb.QB_EINVAL),
                       (8, 0, qb.QB_EINVAL), (9, NUL, qb.QB_EINVAL), (9, ODD, qb.QB_EINVAL),
                       (10, 1, qb.QB_EINVAL), (10, 2, qb.QB_EINVAL)]:
        bad = [v if j == i else a for j, a in enumerate(ok)]
        assert qb.lib.qb_fp8_expert_wgrad(*bad) == want, (i, v)
    # several groups have columns whatever their tokens (fp8_cols_width): none is too few
    several = [F, F, F, F, F, 2, 0, 64, 48, F, 0, 0, NUL]
    assert qb.lib.qb_fp8_expert_wgrad(*several) == qb.QB_EINVAL
