"""GPU tests of include/gdn_train.h at the ends of the number range: the
lowest and the largest finite numbers, infinities and NaNs, in every input,
against the float64 oracle (oracle/train.py) and against the same call
without them."""
import numpy as np
import pytest
import torch

import oracle.train as ora
from gpu_util import DEV, gdn, host
from train_util import DT, Case, check_forward, check_grads

pytestmark = pytest.mark.gpu


def largest(act, sign):
    return sign * torch.finfo(DT[act]).max


def check_step(c):
    """Forward and backward against the oracle."""
    saved = c.saved()
    h, _, so = c.forward(saved)
    check_forward(c, h, so, ora)
    out = c.backward(saved)
    check_grads(c, out, ora)


@pytest.mark.parametrize("C", [64, 66])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_products_with_the_largest_x(act, C):
    """lambda x beta (1 - beta) is in range where lambda x beta is not."""
    c = Case([300, 290], C, act, "f32", seed=62)
    for r, ch, end in ((5, 2, 300), (303, C - 1, 590)):
        c.t["x"][r, ch] = largest(act, 1)
        c.t["b"][r, ch] = 0.875
        c.t["dh"][r, ch] = 2.0
        # nothing behind the row, so that only db meets the large state
        c.t["dh"][r + 1:end, ch] = 0.0
        c.d_state[int(r > 299), ch] = 0.0
    check_step(c)
