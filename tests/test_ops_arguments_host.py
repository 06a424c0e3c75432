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
