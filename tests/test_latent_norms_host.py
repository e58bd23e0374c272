"""The 2-norm bound of the latent attention tests, on the CPU: rounded weights and
outputs stay within it, a tile of keys that is lost, or counted twice, does not."""
import numpy as np
import pytest
import torch

from tests import latent_norms as norms
from tests import latent_reference as ref


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().double().numpy()


def rows(mult, n, L, H, seed):
    rng = np.random.default_rng(seed)
    c, kr = bf16(rng.standard_normal((n, L))), bf16(rng.standard_normal((n, 64)))
    q = bf16(rng.standard_normal((1, H, L + 64)) * mult)
    want, p = ref.absorbed(q, c, kr, 1 / 16)
    return q, c, kr, want, p


@pytest.mark.parametrize("mult", [0.0, 0.05, 1.0, 6.0])
@pytest.mark.parametrize("n,L", [(100, 256), (3000, 512), (20000, 512)])
def test_roundings_stay_within(n, L, mult):
    q, c, kr, want, p = rows(mult, n, L, 4, 1)
    tol = norms.absorbed_bound(q, c, kr, p, want, 1 / 16)
    top = p.max(-1, keepdims=True)
    got = bf16(bf16(p / top) * top @ c)         # weights relative to the largest, as rounded
    assert (np.linalg.norm(got - want, axis=-1) <= tol).all()


@pytest.mark.parametrize("mult", [0.0, 0.05, 1.0])
@pytest.mark.parametrize("n,L,tile", [(300, 256, 32), (3000, 512, 32), (20000, 512, 32)])
def test_a_lost_or_doubled_tile_does_not(n, L, tile, mult):
    q, c, kr, want, p = rows(mult, n, L, 4, 2)
    tol = norms.absorbed_bound(q, c, kr, p, want, 1 / 16)
    for at in (0, n // 2 // tile * tile, n - tile):
        for times in (0.0, 2.0):
            w = p.copy()
            w[..., at:at + tile] *= times
            # (seen by a row for which the tile weighs something: most do)
            assert (np.linalg.norm(bf16(w @ c) - want, axis=-1) > tol).any()
