"""The product kernels of the layer for a few tokens, no GPU: every call's plan
asks for kernels that are built, and every built kernel is asked for by a shape
of the list that the GPU tests run."""
import math
import random

import pytest

import decode_kernels as DK


@pytest.mark.parametrize("fmt", DK.FORMATS)
def test_plans_ask_for_built_kernels(fmt):
    built, rng = DK.built_kernels(), random.Random(fmt)
    step = 32 if fmt.endswith("mx") else 8
    log = lambda lo, hi: int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    for _ in range(20000):
        E = min(256, log(1, 256))
        shape = (min(256, log(1, 256)), step * log(1, (1 << 20) // step), E, min(E, log(1, 256)),
                 step * log(1, (1 << 20) // step), rng.choice([0, 0, 1, 8]))
        p = DK.plan(fmt, shape)
        assert set(DK.kernels_of(fmt, shape)) <= built, shape
        assert p.entries <= 65535 and p.slices <= 65535, shape          # a grid's y and z


def test_every_built_kernel_is_reached():
    reached = {k for fmt in DK.FORMATS for s in DK.KERNEL_SHAPES[fmt] for k in DK.kernels_of(fmt, s)}
    assert reached == DK.built_kernels()
