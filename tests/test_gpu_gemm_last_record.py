"""The product with a packed blob whose last record holds infinite weights: their columns are
infinite with x's sign, in tiles of every size and wherever the last step of k ends."""

import numpy as np
import pytest

from tests.test_gpu_layer_ops import _f64, _gen, _randn, env  # noqa: F401
from tests.test_gpu_prompt_ops import _blob

pytestmark = pytest.mark.gpu

# rows, d_out: tiles of 32, 64, 128 and 256 rows among them
SIZES = [(1, [128]), (5, [384]), (70, [256, 128]), (64, [2176, 2176]), (120, [20480]), (200, [12160]),
         (3001, [4352])]


@pytest.mark.parametrize("rows,d_out", SIZES, ids=[f"{r}x{sum(d)}" for r, d in SIZES])
@pytest.mark.parametrize("d_in", [1, 17, 65, 127, 128, 515])
@pytest.mark.parametrize("fmt", ["fp16", "int4"])
def test_infinite_last_weights(env, rows, d_out, d_in, fmt):  # noqa: F811
    torch, spax, dev = env
    d_out = [n // 128 * 128 for n in d_out]
    L, packed, w = _blob(env, d_in, d_out, fmt, d_in)
    n = sum(d_out)
    rec = packed[(d_in - 1) * int(L.stride_F):d_in * int(L.stride_F)]
    # columns of the first and of the last group of 128, the last one negative
    cols = np.r_[0:128, n - 128:n] if fmt == "int4" else np.array([0, 5, 127, n - 128, n - 1])
    inf = np.where(cols < 128, np.inf, -np.inf) if n > 128 else np.full(len(cols), -np.inf)
    if fmt == "int4":
        words = rec[n // 2:n // 2 + n // 128 * 4].view(torch.float16)   # scale, zero of each group
        words[1] = float("inf")
        words[-1] = -float("inf")
    else:
        rec.view(torch.float16)[torch.tensor(cols, device=dev)] = torch.tensor(
            inf, dtype=torch.float16, device=dev)
    x = _randn(torch, _gen(torch, 3), (rows, (d_in + 7) // 8 * 8), torch.float16)[:, :d_in]
    x[:, -1] = torch.where(x[:, -1] >= 0, 1.0, -1.0).half()
    y = torch.full((rows, n), float("nan"), device=dev)
    a = spax.make_packed_gemm(L, packed, x, y)
    need = spax.spax_packed_gemm_workspace_bytes(a)
    spax.spax_packed_gemm(a, torch.empty(need, dtype=torch.uint8, device=dev) if need else None)
    torch.cuda.synchronize()
    got = _f64(y)
    assert np.array_equal(got[:, cols], _f64(x)[:, -1:] * inf[None])
    rest = np.setdiff1d(np.arange(n), cols)
    assert np.isfinite(got[:, rest]).all()
