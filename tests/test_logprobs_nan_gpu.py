"""Order of the likeliest tokens in rows that hold a NaN, at the first column above all: a NaN ranks
above every number, equal ranks go to the lower index, and every index stays inside the row."""
from __future__ import annotations

import numpy as np
import pytest

from _util import ensure_lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
mnb = ensure_lib()
DEV = torch.device("cuda:0")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def order(x, top):
    """Indices by (NaN first, then the larger value, then the lower index)."""
    nan = np.isnan(x)
    keys = np.where(nan, 0.0, x)
    return np.stack([np.lexsort((np.arange(x.shape[1]), -k, ~n))[:top] for k, n in zip(keys, nan)])


# one part of each kernel shape (49152 columns of one row and of 300), and split rows
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,V", [(6, 1), (6, 5), (6, 300), (6, 9000), (6, 49152), (300, 49152), (6, 50257), (6, 200000)])
def test_nan_at_the_first_column(dtype, M, V):
    r = np.random.default_rng([41, M, V])
    x = r.standard_normal((M, V))
    x[0, 0] = np.nan
    x[1] = np.nan
    x[2, 0] = x[2, V // 2] = x[2, V - 1] = np.nan
    x[3, V // 3] = np.inf
    x[3, 0] = np.nan
    x[4, :] = -np.inf
    x[4, 0] = np.nan
    x[M - 1, 0] = -np.nan
    X = torch.from_numpy(x).to(DEV).to(DT[dtype])
    held = X[:6].double().cpu().numpy()
    for top in sorted({1, min(5, V), min(32, V)}):
        got = mnb.logprobs(X, torch.zeros(M, dtype=torch.int64, device=DEV), top)
        tokens = got.top_tokens.cpu().numpy()
        assert tokens.min() >= 0 and tokens.max() < V
        assert np.array_equal(tokens[:6], order(held, top))
        last = [0, 1, 2, 3, 4, M - 1]
        for t in (got.logprob, got.entropy, got.top_logprobs):
            assert bool(t[last].isnan().all())
