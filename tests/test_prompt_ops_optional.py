"""Arguments that belong to a part that is left out are not read."""

import pytest

import activation_sparse_tiered_amd as spax
from activation_sparse_tiered_amd import _lib
from tests.test_layer_ops_abi import FAKE, MB, N, P, needs_no_gpu
from tests.test_prompt_ops_abi import _gemm


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(residual_stride=-1), dict(residual_stride=1 << 60),
                                dict(residual_stride=3, residual_type=99)])
def test_no_residual(kw):
    a = _gemm(d_in=4096, d_out=(4096,), x=FAKE + 200 * MB, y=FAKE + 201 * MB)
    need = spax.spax_packed_gemm_workspace_bytes(a)
    for name, v in kw.items():
        setattr(a, name, v)
    assert spax.spax_packed_gemm_workspace_bytes(a) == need > 0
    assert _lib.lib.spax_packed_gemm(a, 0, 0, 0) == N, _lib.lib.spax_last_error()   # the workspace
    a.residual, a.residual_type = FAKE + 202 * MB, spax.TYPE_F32
    assert _lib.lib.spax_packed_gemm(a, 0, 0, 0) == P
