"""Latent path, host side (no GPU): refusals before any launch, the frequency
helper, the binding's checks, and the references' own pins."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_143_gb300 import pa
from tests import latent_reference as ref

P = 16  # a fake, aligned device pointer: the calls return before touching it


def latent_pool(**kw):
    d = dict(latent=P, rope=P, scales=None, num_blocks=4, block_size=16, latent_dim=512,
             rope_dim=64, dtype=0)
    d.update(kw)
    return ctypes.byref(pa._LatentPool(*[d[n] for n, _ in pa._LatentPool._fields_]))


BAD_POOLS = [
    (dict(latent=None), pa.PA_ERR_INVALID), (dict(rope=24), pa.PA_ERR_INVALID),
    (dict(num_blocks=-1), pa.PA_ERR_INVALID), (dict(latent_dim=384), pa.PA_ERR_UNSUPPORTED),
    (dict(rope_dim=32), pa.PA_ERR_UNSUPPORTED), (dict(block_size=24), pa.PA_ERR_UNSUPPORTED),
    (dict(dtype=2), pa.PA_ERR_UNSUPPORTED), (dict(dtype=1), pa.PA_ERR_INVALID),
    (dict(num_blocks=1 << 28), pa.PA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_POOLS)
def test_pool_refusals(kw, status):
    L = pa.lib()
    assert L.pa_write_latent(latent_pool(**kw), P, 512, P, 64, None, None, 0, 1.0, P, 1,
                             None) == status
    assert L.pa_read_latent(latent_pool(**kw), P, 1, P, None, 1, 1, P, 512, P, 64, None) == status
    assert L.pa_copy_latent_blocks(latent_pool(**kw), P, P, 1, None) == status


def test_write_latent_refusals():
    L = pa.lib()
    ok = dict(latent=P, ls=512, rope=P, rs=64, pos=None, freq=None, layout=0, factor=1.0, slots=P,
              T=1)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pa_write_latent(latent_pool(), a["latent"], a["ls"], a["rope"], a["rs"], a["pos"],
                                 a["freq"], a["layout"], a["factor"], a["slots"], a["T"], None)

    assert call(T=0) == pa.PA_OK
    for bad in (dict(T=-1), dict(latent=None), dict(latent=24), dict(rope=None), dict(rope=17),
                dict(slots=None), dict(slots=12), dict(ls=513), dict(ls=-8), dict(rs=-1),
                dict(layout=2), dict(pos=P), dict(freq=P), dict(pos=18, freq=P),
                dict(pos=P, freq=P, factor=0.0), dict(pos=P, freq=P, factor=float("nan")),
                dict(pos=P, freq=P, factor=float("inf"))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_read_latent_and_copy_refusals():
    L = pa.lib()
    ok = dict(tab=P, mb=1, start=P, R=1, N=1, c=P, cs=512, kr=P, rs=64)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pa_read_latent(latent_pool(), a["tab"], a["mb"], a["start"], None, a["R"], a["N"],
                                a["c"], a["cs"], a["kr"], a["rs"], None)

    assert call(N=0) == pa.PA_OK
    for bad in (dict(N=-1), dict(R=-1), dict(R=0), dict(mb=-1), dict(tab=None), dict(start=None),
                dict(c=None), dict(c=24), dict(cs=504), dict(cs=516), dict(kr=None), dict(kr=18),
                dict(rs=62), dict(rs=65)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert L.pa_copy_latent_blocks(latent_pool(), P, P, 0, None) == pa.PA_OK
    assert L.pa_copy_latent_blocks(latent_pool(), P, P, -1, None) == pa.PA_ERR_INVALID
    assert L.pa_copy_latent_blocks(latent_pool(), None, P, 1, None) == pa.PA_ERR_INVALID


def test_rope_refusals():
    L = pa.lib()
    ok = dict(x=P, xt=256, xh=64, out=32, ot=256, oh=64, pos=P, T=3, H=4, D=64, freq=P, rot=64,
              layout=0, factor=1.0)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pa_rope(a["x"], a["xt"], a["xh"], a["out"], a["ot"], a["oh"], a["pos"], a["T"],
                         a["H"], a["D"], a["freq"], a["rot"], a["layout"], a["factor"], None)

    assert call(T=0) == pa.PA_OK
    assert call(rot=0, freq=None, out=P) == pa.PA_OK  # in place, nothing turned
    for bad in (dict(T=-1), dict(H=0), dict(D=0), dict(rot=-2), dict(rot=66), dict(layout=3),
                dict(factor=0.0), dict(factor=float("nan")), dict(x=None), dict(out=None),
                dict(pos=None), dict(freq=None), dict(x=17), dict(pos=18), dict(xt=-1),
                dict(oh=0), dict(ot=64), dict(oh=32), dict(out=P, ot=512), dict(out=P, oh=65)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert call(rot=31) == pa.PA_ERR_UNSUPPORTED
    assert call(D=512, rot=258, xh=512, oh=512, xt=2048, ot=2048) == pa.PA_ERR_UNSUPPORTED
    assert call(H=1, D=32776, xt=40000, ot=40000) == pa.PA_ERR_UNSUPPORTED


def test_rope_sizes_whose_products_pass_64_bits():
    """Strides that no memory holds are refused, not multiplied; so are rows that
    overlap by them."""
    L = pa.lib()

    def call(T, H, D, xt, xh, ot, oh):
        return L.pa_rope(P, xt, xh, 32, ot, oh, P, T, H, D, P, 2, 0, 1.0, None)

    top = 2 ** 31 - 1
    for a in ((2, 3, 64, 64, 64, 64, 1 << 62), (3, 2, 64, 64, 64, 1 << 62, 64),
              (2, 2, 64, 1 << 62, 64, 128, 64), (2, 2, 64, 128, 1 << 38, 128, 64),
              (top, top, 1, 0, 0, (1 << 38) - 1, (1 << 38) - 1), (top, top, 1, 0, 0, top - 1, 1)):
        assert call(*a) == pa.PA_ERR_INVALID, a
    assert call(1, top, 32768, 0, 0, 0, 32768) == pa.PA_ERR_UNSUPPORTED


def test_binding_checks_without_a_device():
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not a CUDA tensor
        pa.rope(x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(4))
    with pytest.raises(ValueError):
        pa.rope(x, x, torch.zeros(3, dtype=torch.int32), torch.zeros(4))
    lat, rot = torch.zeros(2, 16, 256, dtype=torch.uint8), torch.zeros(2, 16, 64)
    with pytest.raises(ValueError):  # E4M3 without scales
        pa.LatentPool(lat, rot)
    with pytest.raises(ValueError):  # bf16 with scales
        pa.LatentPool(lat.bfloat16(), rot, torch.zeros(2, 16))
    with pytest.raises(TypeError):
        pa.LatentPool(lat.float(), rot)
    with pytest.raises(ValueError):
        pa.LatentPool(lat.bfloat16(), rot[:1])


def test_rope_frequencies():
    f, a = pa.rope_frequencies(64)
    assert f.dtype == torch.float32 and f.numel() == 32 and a == 1.0
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-7)
    lin, _ = pa.rope_frequencies(64, scaling="linear", stretch=4.0)
    np.testing.assert_allclose(lin.numpy(), f.numpy() / 4, rtol=1e-6)
    b, _ = pa.rope_frequencies(64, scaling="base", stretch=8.0)
    assert b[0] == f[0]
    np.testing.assert_allclose(b[-1] * 8, f[-1], rtol=1e-5)
    p, a = pa.rope_frequencies(64, scaling="by_parts", stretch=8.0, original_context=4096)
    turns = 4096 * f.numpy().astype(np.float64) / (2 * np.pi)
    fast, slow = turns > 32, turns < 1
    assert fast.any() and slow.any() and (~fast & ~slow).any()
    np.testing.assert_allclose(p.numpy()[fast], f.numpy()[fast], rtol=1e-7)
    np.testing.assert_allclose(p.numpy()[slow], f.numpy()[slow] / 8, rtol=1e-6)
    assert np.all(np.diff(p.numpy()) < 0) and abs(a - (1 + 0.1 * np.log(8))) < 1e-12
    same, a = pa.rope_frequencies(64, scaling="by_parts", stretch=1.0)
    np.testing.assert_allclose(same.numpy(), f.numpy(), rtol=1e-7)
    assert a == 1.0
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, stretch=0.5),
                dict(rot_dim=64, scaling="x"), dict(rot_dim=2, scaling="base"),
                dict(rot_dim=64, scaling="by_parts", fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            pa.rope_frequencies(**bad)


def test_reference_quantiser_matches_torch_e4m3():
    """The reference's E4M3 rounding and decoding against torch's own type."""
    x = torch.linspace(-448, 448, 40001, dtype=torch.float64)
    x = torch.cat((x, x / 4096, torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 464.0])))
    want = x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double().numpy()
    # float() of these points is exact or far from a tie, so torch's rounding is the reference's
    np.testing.assert_array_equal(ref.e4m3_round(x.float().double().numpy()), want)
    codes = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(
        ref.e4m3_values(codes), torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())
    assert ref.token_scale(np.array([448.0])) == 1.0
    assert ref.token_scale(np.array([448.5])) == 2.0
    assert ref.token_scale(np.array([0.0, -0.0])) == 1.0
    assert ref.token_scale(np.array([np.inf, -3.5, np.nan])) == 2.0 ** -7
    assert ref.token_scale(np.array([1e-40])) == 2.0 ** -60


def test_reference_absorbed_equals_expanded():
    """The two forms agree: keys [W_k c ; k_r] and values W_v c attended to in
    full, against the query moved into the latent space."""
    rng = np.random.default_rng(5)
    H, dn, dv, L, N, Tq = 3, 8, 8, 16, 11, 4
    c, kr = rng.standard_normal((N, L)), rng.standard_normal((N, ref.ROPE))
    wk, wv = rng.standard_normal((H, dn, L)), rng.standard_normal((H, dv, L))
    q = rng.standard_normal((Tq, H, dn + ref.ROPE))
    full, _ = ref.expanded(q, np.einsum("hdl,nl->nhd", wk, c), kr,
                           np.einsum("hdl,nl->nhd", wv, c), 0.2)
    qa = np.concatenate((np.einsum("thd,hdl->thl", q[..., :dn], wk), q[..., dn:]), -1)
    o, _ = ref.absorbed(qa, c, kr, 0.2)
    np.testing.assert_allclose(np.einsum("thl,hdl->thd", o, wv), full, atol=1e-12)


def test_latent_forward_refusals():
    L = pa.lib()
    qsl, seq = np.array([0, 1, 3], np.int32), np.array([40, 50], np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    ok = dict(q=P, out=P, qsl=P, seq=P, qh=qsl, sh=seq, tab=P, mb=4, R=2, T=3, H=16, pool={},
              scale=0.1, causal=1, ws=None, wb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pa_latent_forward(a["q"], a["out"], a["qsl"], a["seq"], ptr(a["qh"]),
                                   ptr(a["sh"]), a["tab"], a["mb"], a["R"], a["T"], a["H"],
                                   latent_pool(**a["pool"]), a["scale"], a["causal"], a["ws"],
                                   a["wb"], None)

    i = lambda *v: np.array(v, np.int32)
    for bad in (dict(), dict(ws=P, wb=4096),  # a workspace is required, of the whole size
                dict(ws=24, wb=1 << 30), dict(ws=None, wb=1 << 30), dict(q=None), dict(q=24),
                dict(out=None), dict(out=40), dict(qsl=None), dict(seq=None), dict(qh=None),
                dict(sh=None), dict(tab=None), dict(mb=-1), dict(mb=3), dict(R=-1), dict(T=-1),
                dict(T=4), dict(H=0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(causal=2),
                dict(qh=i(1, 1, 3)), dict(qh=i(0, 4, 3)), dict(sh=i(40, 1)), dict(sh=i(0, 50)),
                dict(sh=i(65, 50)), dict(pool=dict(num_blocks=0)), dict(R=0)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert call(R=0, T=0) == pa.PA_OK
    assert call(T=0, qh=i(0, 0, 0)) == pa.PA_OK
    assert call(pool=dict(latent_dim=128)) == pa.PA_ERR_UNSUPPORTED
    assert call(H=1 << 30) == pa.PA_ERR_UNSUPPORTED  # rows past 32-bit coordinates
    assert pa.latent_workspace_size(0, 512) == 0 and pa.latent_workspace_size(16, 100) == 0


def test_latent_prefill_refusals():
    L = pa.lib()
    i = lambda *v: np.array(v, np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(ctypes.c_void_p)
    ok = dict(q=P, qt=768, qh=192, k=P, kt=512, kh=128, kr=P, rt=64, v=P, vt=512, vh=128, out=P,
              qsl=P, ksl=P, qhost=i(0, 1, 3), khost=i(0, 4, 9), R=2, T=3, Tk=9, H=4, dn=128,
              dr=64, dv=128, scale=0.1, causal=1)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pa_latent_prefill(
            a["q"], a["qt"], a["qh"], a["k"], a["kt"], a["kh"], a["kr"], a["rt"], a["v"], a["vt"],
            a["vh"], a["out"], a["qsl"], a["ksl"], ptr(a["qhost"]), ptr(a["khost"]), a["R"],
            a["T"], a["Tk"], a["H"], a["dn"], a["dr"], a["dv"], a["scale"], a["causal"], None)

    for bad in (dict(R=-1), dict(T=-1), dict(Tk=-1), dict(H=0), dict(scale=0.0),
                dict(scale=float("nan")), dict(causal=3), dict(qhost=None), dict(khost=None),
                dict(qsl=None), dict(ksl=None), dict(T=4), dict(Tk=8), dict(qhost=i(0, 4, 3)),
                dict(khost=i(0, 10, 9)), dict(qhost=i(1, 1, 3)), dict(q=None), dict(q=24),
                dict(out=None), dict(out=24), dict(k=None), dict(v=None), dict(kr=None),
                dict(k=24), dict(v=24), dict(kr=24), dict(qt=770), dict(qh=0), dict(kt=-8),
                dict(kh=132), dict(vt=0), dict(vh=4), dict(rt=60), dict(R=0)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert call(R=0, T=0, Tk=0) == pa.PA_OK
    assert call(T=0, qhost=i(0, 0, 0)) == pa.PA_OK
    for bad in (dict(dn=64), dict(dr=32), dict(dv=64)):
        assert call(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    n = 40000
    assert call(R=n, T=n, Tk=0, qhost=np.arange(n + 1, dtype=np.int32),
                khost=np.zeros(n + 1, np.int32)) == pa.PA_ERR_UNSUPPORTED
