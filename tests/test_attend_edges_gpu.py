"""pld_attend (HIP, gfx950) at the edges of its arguments: scales so small
that they vanish in 32 bits. Tolerances are test_attend_gpu.py's."""

from __future__ import annotations

import numpy as np
import pytest

from prompt_lookup_gram_amd import binding as B
from test_attend_gpu import Case, check, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [1e-45, -1e-45, 1e-39, 1e-30])
@pytest.mark.parametrize("rows", [1, 4, 20])
def test_scales_that_vanish_weigh_every_position_the_same(cache, scale, rows):
    # (1e-45 times a cell scale below 1 is 0; masked scores stay out all the same)
    check([70, 33, 300], [rows - 1, 0, rows // 2], rows, scale=scale, cache=cache, window=40,
          seed=20)
