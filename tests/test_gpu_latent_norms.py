"""GPU tests of both forms of latent attention by the 2-norm of each output row's
error, which sees a tile of keys that is lost or counted twice (tests/latent_norms.py)."""
import numpy as np
import pytest

from paged_kv_cache_143_gb300 import pa
from tests import latent_norms as norms
from tests import latent_reference as ref
from tests.test_gpu_latent_attention import Batch
from tests.test_gpu_latent_prefill import DN, Chunks

pytestmark = pytest.mark.gpu

ABSORBED = [  # seq_lens, q_lens, H, L, B, mult
    ([3000, 70, 640], [1, 1, 5], 16, 512, 16, 0.0), ([3000, 70, 640], [1, 1, 5], 16, 512, 16, 0.05),
    ([3000, 70, 640], [1, 1, 5], 16, 256, 16, 1.0), ([20000], [1], 16, 512, 32, 0.05),
    ([20000], [2], 64, 256, 64, 1.0), ([4000, 4000, 300], [1, 4, 40], 24, 512, 64, 0.3),
    ([900] * 40, [1] * 40, 128, 512, 64, 1.0), ([700] * 200, [1] * 200, 8, 256, 16, 1.0),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(ABSORBED)))
def test_absorbed(cuda_device, case, fp8):
    seqs, q_lens, H, L, B, mult = ABSORBED[case]
    b = Batch(seqs, q_lens, H, L, B, fp8, cuda_device, seed=70 + case, mult=mult)
    b.run()
    assert pa.get_error() == pa.PA_OK
    lat, rot = ref.pool_rows(b.pool)
    for r in range(len(seqs)):
        a, e = b.qsl[r], b.qsl[r + 1]
        at = ref.slots_of(b.tab, r, seqs[r], B)
        q, c, kr = ref.f64(b.q[a:e]), lat[at], rot[at]
        want, p = ref.absorbed(q, c, kr, b.scale)
        scales = ref.f64(b.pool.scales).reshape(-1)[at] if fp8 else None
        tol = norms.absorbed_bound(q, c, kr, p, want, b.scale, scales)
        err = np.linalg.norm(ref.f64(b.out[a:e]) - want, axis=-1)
        assert (err <= tol).all(), (r, (err / tol).max())


EXPANDED = [  # q_lens, k_lens, H, mult
    ([200, 300], [900, 300], 2, 0.0), ([200, 300], [900, 300], 2, 1.0), ([5], [3000], 1, 0.1),
    ([300], [5000], 1, 0.5), ([700, 40], [2100, 2000], 3, 1.0), ([5, 7], [9000, 4000], 4, 0.0),
]


@pytest.mark.parametrize("case", range(len(EXPANDED)))
def test_expanded(cuda_device, case):
    q_lens, k_lens, H, mult = EXPANDED[case]
    b = Chunks(q_lens, k_lens, H, cuda_device, seed=80 + case, mult=mult)
    b.run()
    assert pa.get_error() == pa.PA_OK
    for r in range(len(q_lens)):
        a, e, c, d = b.qsl[r], b.qsl[r + 1], b.ksl[r], b.ksl[r + 1]
        q, k, kr, v = (ref.f64(t) for t in (b.q[a:e], b.k[c:d], b.kr[c:d], b.v[c:d]))
        want, p = ref.expanded(q, k, kr, v, b.scale)
        for h in range(H):
            s = np.abs(q[:, h, :DN]) @ np.abs(k[:, h]).T + np.abs(q[:, h, DN:]) @ np.abs(kr).T
            tol = norms.bound(p[:, h], v[:, h], want[:, h], 2.0 ** -20 * b.scale * s.max(-1))
            err = np.linalg.norm(ref.f64(b.out[a:e, h]) - want[:, h], axis=-1)
            assert (err <= tol).all(), (r, h, (err / tol).max())
