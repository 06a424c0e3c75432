"""Arguments of the torch calls that are no tensors, or fail when they are read (host only)."""
from __future__ import annotations

import numpy as np
import pytest

from _util import ensure_lib

mnb = ensure_lib()
torch = pytest.importorskip("torch")


def test_an_error_in_keep16_is_passed_on():
    class Odd:
        def __bool__(self):
            raise ZeroDivisionError("of the caller")
    x, w = torch.zeros(4, 64, dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    with pytest.raises(ZeroDivisionError, match="of the caller"):
        mnb.rmsnorm(x, w, fmt=mnb.MNB_MX_FP8, keep16=Odd())


@pytest.mark.parametrize("bad", [None, 3, np.zeros((4, 64), np.float16), [[1.0]]])
def test_what_is_no_tensor_is_a_type_error(bad):
    x, w = torch.zeros(4, 64, dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    for call in (lambda: mnb.mx_quantize(bad), lambda: mnb.rmsnorm(bad, w), lambda: mnb.logprobs(bad),
                 lambda: mnb.rmsnorm(x, bad), lambda: mnb.logprobs(x, bad if bad is not None else 7)):
        with pytest.raises(TypeError, match="tensor"):
            call()
