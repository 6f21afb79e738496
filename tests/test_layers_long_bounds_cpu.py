"""The bounds of tests/test_layers_long_gpu.py see a lost, doubled or misplaced
piece: the 64-bit reference with such a mistake planted in it is out of them."""
import pytest
import torch

from . import test_layers_long_gpu as G

N, LO = 70001, 64 * 500  # the tile of positions LO .. LO + 63


def lost(j):
    return torch.cat([j[:LO], j[LO + 64:]])


def doubled(j):
    return torch.cat([j, j[LO:LO + 64]])


def misplaced(j):
    return torch.cat([j[:LO], j[LO + 64:LO + 128], j[LO + 64:]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mistake", [lost, doubled, misplaced])
def test_a_mistaken_tile_is_out_of_bounds(mistake, dtype):
    gen = torch.Generator().manual_seed(0)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v, table, shown = G.build(gen, [N], 1, 64, 128, dt)
    q = torch.randn((1, 1, 4, 128), generator=gen).to(dt)
    mass = torch.rand((1, 1, table.shape[1] * 64), generator=gen)
    args = (q, k, v, table, shown, [N], 128 ** -0.5, mass)
    ref, wrong = G.reference(*args), G.reference(*args, keep=mistake)
    lims = G.bounds(q, k, 128 ** -0.5, 60, 300, ref, mass)
    lse, drawn = (float(((wrong[i] - ref[i]).abs() / lims[i].clamp_min(1e-300)).max()) for i in (1, 2))
    assert drawn > 100  # whole weights
    assert lse > 1 or mistake is misplaced  # that one puts as much weight in as it takes out
    # The same reference is within them, of course.
    assert all(float(((a - b).abs() / lim.clamp_min(1e-300)).max()) == 0 for a, b, lim in zip(ref, ref, lims))
