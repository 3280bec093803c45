"""The splits of a slot added up a warp or a CTA a row, up to four records at once or in turn, by the batch's size and its splits:
the same bits whichever does it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_87_window import Case as WindowCase
from tests.test_gpu_94_quant_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [512, 640, 1500, 1664])     # 4, 5, 12 and 13 splits of 128
def test_a_slot_s_bits_do_not_depend_on_who_adds_them_up(gpu_lib, most):
    k3 = gpu_lib
    g = np.random.default_rng(most)
    c = Case([most] + [int(x) for x in g.integers(1, most, 43)], seed=most).stale()
    whole = c.run(k3, split=128, max_ctx=most)
    c.check(whole)
    for n in (39, 24, 23, 17, 16, 5):
        slots = [int(x) for x in g.permutation(44)[:n]]
        assert torch.equal(c.run(k3, split=128, max_ctx=most, slots=slots), whole[slots]), n


@pytest.mark.parametrize("most", [512, 1500, 2100])
def test_the_same_over_the_bf16_cache(gpu_lib, most):
    g = np.random.default_rng(most + 1)
    lens = [most] + [int(x) for x in g.integers(1, most, 43)]
    c = WindowCase(3, lens, 44)
    whole = c.decode(10 ** 6, 0, 128)
    for n in (39, 23, 17, 9):
        slots = g.permutation(44)[:n]
        assert torch.equal(c.decode(10 ** 6, 0, 128, slots=slots), whole[torch.from_numpy(slots).cuda()]), n
