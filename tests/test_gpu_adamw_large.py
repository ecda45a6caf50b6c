"""AdamW steps of more than 2,048 tiles, whose master copies and 32-bit states go past the caches: every
tensor, state and packed form by the definition of tests/test_gpu_adamw.py, for A and B of small ranks and
large, a vector, and a group that makes no step, with norms and without."""

import numpy as np
import pytest

from test_gpu_adamw import Case

pytestmark = pytest.mark.gpu

# tiles: 512 rows (columns) of ranks up to 4, 256 up to 16, 128 up to 32, 64 above, and 4,096 values of a vector
SHAPES = [x for r in (1, 2, 3, 4, 5, 7, 8, 11, 16, 17, 24, 32, 33, 50, 64) for side, g in ((4160, r % 4), (8256, (r + 1) % 4))
          for x in (("A", side, r, g), ("B", r, side, (g + 2) % 4))] + [("plain", 1, 100003, 0), ("plain", 7, 12800, 3)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [False, True])
def test_steps_past_the_caches(clip, bits):
    print("[case] adamw large", clip, bits, flush=True)
    c = Case(SHAPES, 4, bits, 21)
    assert c.opt.tiles.shape[0] > 2048
    rng = np.random.default_rng(5)
    for active in (None, [1, 1, 0, 1]):
        before = c.values()
        norms = c.norms(before, active)
        got = c.step(active, clip)
        c.steps += 1 if active is None else np.asarray(active, np.int32)
        assert np.array_equal(c.opt.steps.cpu().numpy(), c.steps)
        if clip:
            assert (np.abs(got.double().cpu().numpy() - norms) <= 2.0 ** -23 * norms).all()
        c.check(before, norms, active, clip)
        scale = float(rng.uniform(-1, 1))
        for t in c.tensors:  # the next step's gradients
            t.grad.mul_(scale).add_(0.002)
