"""Column ranges of one wide buffer are apart: the operators around the linear
take them as inputs and outputs of a call, and refuse ranges that meet."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
from test_ops_cpu import A, DEVICE, UNSUP, combine, grouped, lora, norm  # noqa: E402


def at(column, size=2, base=A(20)):
    return base + column * size


# rows of 64 values side by side in a buffer whose rows hold 256 values
APART = [
    (norm, dict(x=at(0), ldx=256, sum=at(64), lds=256, y=at(128), ldy=256, res=at(192), ldr=256)),
    (norm, dict(x=at(64), ldx=256, sum=at(64), lds=256, y=at(0), ldy=256)),
    # 512-byte rows that hold x, the bytes and the codes of a row
    (norm, dict(x=at(0), ldx=256, xq=at(64), ldq=512, xc=at(128), ldc=512)),
    (grouped, dict(x=at(0), ldx=512, y=at(256), ldy=512)),
    (grouped, dict(x=at(64), ldx=512, y=at(0), ldy=512)),
    (combine, dict(ys=at(64), ldys=128, y=at(0), ldy=128)),
    (lora, dict(x=at(0), ldx=256, base=at(96), ldb=256, y=at(160), ldy=256)),
    (lora, dict(x=at(0), ldx=256, base=at(96), ldb=256, y=at(96), ldy=256)),
    # a range that ends where the next row's begins
    (lora, dict(x=at(160), ldx=256, base=at(0), ldb=256, y=at(96), ldy=256)),
]
MEET = [
    (norm, dict(x=at(0), ldx=256, sum=at(56), lds=256)),
    (norm, dict(x=at(64), ldx=256, sum=at(8), lds=256)),
    (norm, dict(x=at(0), ldx=256, xq=at(56), ldq=512)),
    (norm, dict(x=at(216), ldx=256, y=at(256), ldy=256)),          # x runs into the next row
    (norm, dict(x=at(0), ldx=256, sum=at(64), lds=248)),           # another pitch
    (grouped, dict(x=at(0), ldx=512, y=at(248), ldy=512)),
    (combine, dict(ys=at(64), ldys=128, y=at(8), ldy=128)),
    (lora, dict(x=at(0), ldx=256, base=at(96), ldb=256, y=at(152), ldy=256)),
    (lora, dict(x=at(0), ldx=256, base=at(128), ldb=256, y=at(88), ldy=256)),
]


@pytest.mark.parametrize("call,kw", APART)
def test_apart(call, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the fake addresses must not reach a GPU")
    assert call(**kw) == DEVICE


@pytest.mark.parametrize("call,kw", MEET)
def test_meet(call, kw):
    assert call(**kw) == UNSUP
