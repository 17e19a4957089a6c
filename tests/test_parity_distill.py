"""Parity of distillation's loss and gradient with the 64-bit definition.  Tolerances: a loss is a difference of
logarithms and sums of some 2^-22 each (exponentials by the SFU), relative to the size of its terms; a gradient's
q and p have relative errors of 2e-6 (the exponent's rounding, 2^-24 of |z - max| / τ up to 30, and the sums'), and
a bfloat16 one its half step beside that."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import training_ref as ref

from helpers import to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def case(rows, V, K, io="f32", tio="f32", tau=1.0, seed=0, pad=0, missing=0.2):
    g = torch.Generator("cuda").manual_seed(seed + 13 * V + K)
    z = (2.5 * torch.randn(rows, V + pad, generator=g, device="cuda")).to(DT[io])[:, :V]
    ids = torch.randint(V, (rows, K), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(rows, K, generator=g, device="cuda") < missing] = -1
    t = (3 * torch.randn(rows, K, generator=g, device="cuda")).to(DT[tio])
    return torch.randn(rows, generator=g, device="cuda"), z, ids, t, tau


def check(dloss, z, ids, t, tau, **kw):
    vl, vd = ref.distill(to_host(z), ids.cpu().numpy().astype(np.int64), to_host(t), tau, to_host(dloss))
    alone = ss.ss_distill(z, ids, t, temperature=tau)
    dtype, src = z.dtype, to_host(z)
    loss, d = ss.ss_distill_grad(dloss, z, ids, t, temperature=tau, **kw)
    assert torch.equal(alone, loss)
    at = np.clip(ids.cpu().numpy(), 0, src.shape[1] - 1)
    far = np.abs(np.take_along_axis(src, at, 1) - src.max(1, keepdims=True)).max(1, initial=0.0)
    size = 1 + np.abs(vl) + far / tau                                    # (of the loss's terms)
    assert np.all(np.abs(to_host(loss) - vl) <= 2e-6 * size)
    # q and p behind each value of the gradient
    g = np.abs(to_host(dloss))[:, None] / tau
    q = np.exp(src / tau - src.max(1, keepdims=True) / tau)
    q = q / q.sum(1, keepdims=True) * (vd != 0).any(1, keepdims=True)
    terms = g * q + np.abs(vd - np.sign(to_host(dloss))[:, None] * g * q)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(to_host(d) - vd) <= 4e-6 * terms + half * np.abs(vd) + 1e-37)
    return loss, d


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V,K", [(1, 1, 1), (2, 3, 2), (3, 7, 16), (5, 100, 4), (1, 1000, 64), (7, 4097, 33), (2, 50257, 16),
                                      (700, 1023, 5), (1, 128000, 128), (3, 65536, 1024), (500, 9000, 8)])
def test_sizes(io, rows, V, K):
    check(*case(rows, V, K, io))


@pytest.mark.parametrize("tau", [0.5, 2.0, 7.0])
@pytest.mark.parametrize("io,tio", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_temperatures_and_types(io, tio, tau):
    check(*case(9, 5000, 20, io, tio, tau))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strides(io, pad):
    dloss, z, ids, t, tau = case(6, 3001, 10, io, pad=pad)
    out = torch.full((6, 3001 + 8), 7.0, dtype=DT[io], device="cuda")
    for at in (0, 1, 8):                                     # rows against the 16 bytes as the logits' and otherwise
        _, d = check(dloss, z, ids, t, tau, dlogits=out[:, at:at + 3001])
    assert (out[:, 0:8] != 7.0).any() and out.shape == (6, 3009)
    out = torch.full((6, 3020), 7.0, dtype=DT[io], device="cuda")
    check(dloss, z, ids, t, tau, dlogits=out[:, 5:3006])
    assert (out[:, :5] == 7).all() and (out[:, 3006:] == 7).all()
    check(dloss[:1].expand(6), z, ids, t, tau)
    check(dloss, z[:1].expand(6, 3001), ids, t, tau)
    wide = torch.zeros(6, 30, dtype=torch.int32, device="cuda")
    wide[:, 4:14] = ids
    check(dloss, z, wide[:, 4:14], t, tau)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(4, 100000), (400, 5000)])
def test_in_place(io, rows, V):
    dloss, z, ids, t, tau = case(rows, V, 40, io)
    want = ss.ss_distill_grad(dloss, z, ids, t)
    loss, d = ss.ss_distill_grad(dloss, z, ids, t, dlogits=z)
    assert d is z and torch.equal(d, want[1]) and torch.equal(loss, want[0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 70000])
def test_the_same_column_twice(io, V):
    dloss, z, ids, t, tau = case(8, V, 12, io, missing=0.0)
    ids[:, 3] = ids[:, 0]
    ids[:, 11] = ids[:, 0]
    ids[1] = 7
    ids[2] = V - 1
    check(dloss, z, ids, t, tau)


@pytest.mark.parametrize("V", [640, 60000])
def test_rows_without_weight(V):
    dloss, z, ids, t, tau = case(7, V, 6)
    ids[0] = -1
    t[1] = -INF
    t[2, :5] = -INF
    ids[2, 5] = 3
    dloss[0], dloss[1] = NAN, INF
    z[0], z[1, 5] = NAN, INF                                 # not read
    loss, d = ss.ss_distill_grad(dloss, z, ids, t)
    assert loss[0] == 0 and loss[1] == 0 and not d[:2].any()
    check(dloss[2:], z[2:], ids[2:], t[2:], tau)
    loss, d = ss.ss_distill_grad(dloss, z, ids[:, :0], t[:, :0])
    assert not loss.any() and not d.any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_masked_logits(io):
    """Columns of -inf or of the type's lowest value have no probability; a whole row of the lowest is even."""
    dloss, z, ids, t, tau = case(4, 500, 5, io, tau=0.5, missing=0.0)
    ids[:] = torch.arange(5, device="cuda", dtype=torch.int32)
    z[0, 100:], z[1, 100:] = -INF, torch.finfo(DT[io]).min
    z[2] = torch.finfo(DT[io]).min
    loss, d = check(dloss, z[:], ids, t, tau)
    assert not d[:2, 100:].any()
    z[3, 2] = -INF                                           # under an entry
    loss, d = ss.ss_distill_grad(dloss, z, ids, t, temperature=tau)
    assert loss[3] == INF and torch.isfinite(d).all()


def test_non_finite_rows_stay_alone():
    dloss, z, ids, t, tau = case(6, 900, 5, missing=0.0)
    z[0, 3], z[1, 4], z[2], t[3, 1] = NAN, INF, -INF, NAN
    loss, d = ss.ss_distill_grad(dloss, z, ids, t)
    assert torch.isnan(loss[:4]).all() and torch.isfinite(loss[4:]).all() and torch.isfinite(d[4:]).all()
    check(dloss[4:], z[4:], ids[4:], t[4:], tau)


def test_ids_out_of_range_are_reported_and_left_out():
    dloss, z, ids, t, tau = case(3, 200, 6, missing=0.0)
    bad = ids.clone()
    bad[1, 2], bad[2, 0], ids[1, 2], ids[2, 0] = 200, 2 ** 31 - 1, -1, -1
    got = ss.ss_distill_grad(dloss, z, bad, t)
    assert ss.device_error(clear=True) == 4
    want = ss.ss_distill_grad(dloss, z, ids, t)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_past_32_bit_offsets():
    rows, V = 34000, 65536                                    # 2.2e9 elements
    z = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    z[-1] = torch.randn(V, device="cuda").to(torch.bfloat16)
    ids = torch.arange(4, dtype=torch.int32, device="cuda").expand(rows, 4).contiguous()
    t = torch.zeros(rows, 4, device="cuda")
    dloss = torch.ones(rows, device="cuda")
    loss, d = ss.ss_distill_grad(dloss, z, ids, t)
    vl, vd = ref.distill(to_host(z[-1:]), ids[-1:].cpu().numpy(), to_host(t[-1:]), 1.0, np.ones(1))
    assert abs(float(loss[-1]) - vl[0]) <= 2e-5 and np.all(np.abs(to_host(d[-1:]) - vd) <= 2.0 ** -8 * np.abs(vd) + 1e-9)
    assert torch.equal(d[0], d[-2])


def test_refusals():
    dloss, z, ids, t, tau = case(3, 64, 4)
    with pytest.raises(ss.SelscanError):
        ss.ss_distill(z, ids, t, temperature=0.0)
    with pytest.raises(TypeError):
        ss.ss_distill(z, ids.long(), t)
    with pytest.raises(TypeError):
        ss.ss_distill(z.half(), ids, t)
    with pytest.raises(ValueError):
        ss.ss_distill(z, ids, t[:, :3])
    with pytest.raises(ValueError):
        ss.ss_distill_grad(dloss[:2], z, ids, t)
    with pytest.raises(ValueError):
        ss.ss_distill(z.t(), ids, t)
    with pytest.raises(ss.SelscanError):
        ss.ss_distill_grad(dloss, z[:, :60], ids, t, dlogits=z[:, 2:62])
