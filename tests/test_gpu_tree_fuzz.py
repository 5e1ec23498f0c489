"""Random shapes of the tree attention against the 64-bit reference (tolerances of test_gpu_tree), small
and odd, over the whole range of the call's sizes; and runs of calls that share tensors."""
import numpy as np
import pytest
import torch

from test_gpu_append import swa  # noqa: F401  (the fixture)
from test_gpu_tree import KINDS, Case

pytestmark = pytest.mark.gpu


def shape(rng):
    B = int(rng.integers(1, 7))
    Hkv, G = int(rng.choice([1, 2, 3, 5])), int(rng.choice([1, 2, 3, 4, 7, 16, 33]))
    ns = [int(rng.choice([0, 1, 2, 7, 31, 32, 33, 64, 100, 129, 255, 256], p=[.05, .15, .1, .1, .1, .1, .1, .1, .05, .05, .05, .05])) for _ in range(B)]
    ns = [min(n, 1 + 600 // (Hkv * G)) for n in ns]
    bases = [int(rng.choice([0, 1, 63, 64, 127, 128, 129, 255, 511, int(rng.integers(0, 1500))])) for _ in range(B)]
    return dict(ns=ns, bases=bases, Hq=Hkv * G, Hkv=Hkv, d=int(rng.choice([64, 128])), page=1 << int(rng.integers(0, 9)),
                W=int(rng.choice([1, 2, 50, 64, 128, 300, 5000])), S=int(rng.choice([0, 0, 1, 64, 130, 700])),
                routed=float(rng.choice([0, 0.1, 0.5, 1])), deep=float(rng.choice([0.0, 0.5, 0.9, 1.1])))


@pytest.mark.parametrize("seed", range(36))
def test_random_shapes(swa, seed):
    rng = np.random.default_rng(1000 + seed)
    c = Case(kind=KINDS[seed % 3], seed=seed, pad=int(rng.integers(0, 4)), **shape(rng))
    got = c.run(swa)
    assert swa.get_device_error() == 0
    c.check(got)


def test_one_workspace_through_calls_of_other_sizes(swa):
    """What one call leaves in the workspace does not reach the next."""
    cases = [Case([30, 4], [900, 77], 6, 2, 128, 16, kind, 64, routed=0.4, seed=i) for i, kind in enumerate(KINDS)]
    cases += [Case([1] * 9, list(range(0, 900, 100)), 2, 1, 64, 8, kind, 5000, seed=9) for kind in KINDS]
    most = max(swa.decode_tree_workspace(c.T, len(c.lens), c.q.shape[1], c.pages[0].shape[2], c.d, c.dtype) for c in cases)
    ws = torch.full((most,), 255, dtype=torch.uint8, device="cuda")
    alone = [c.run(swa) for c in cases]
    for _ in range(2):
        for c, want in zip(cases, alone):
            got = c.run(swa, workspace=ws)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert swa.get_device_error() == 0


def test_shared_prefix_pages(swa):
    """Sequences whose tables name the same pages, as forks have them."""
    c = Case([8, 8, 8], [320, 320, 320], 4, 2, 128, 32, "bf16", 100, routed=0.5, seed=40)
    c.table[1:, :10] = c.table[0, :10]
    c.check(c.run(swa))
