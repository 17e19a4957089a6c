"""Parity of the residual norm (in the input's type and in 8 bits) with the 64-bit definition.
Tolerances: float32 relative L2 1e-6 (a sum of squares and four roundings); bfloat16 the half step of
its rounding; 8 bits: the code is that of a neighbour of y/scale that single-precision rounding cannot
tell from it, so the decoded value is within half a step and 1e-5 of a step."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref

from helpers import rel_l2, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()


def inputs(rows, D, io, res, seed=0, pad=0):
    g = torch.Generator("cuda").manual_seed(seed + 7 * D)
    x = torch.randn(rows, D + pad, generator=g, device="cuda").to(DT[io])[:, :D]
    r = None if res is None else (2 * torch.randn(rows, D + pad, generator=g, device="cuda")).to(DT[res])[:, :D]
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    return x, r, w


def want(x, r, w, eps=1e-5):
    return ref.norm(to_host(x), None if r is None else to_host(r), to_host(w), eps)


def close(t, v, what):
    h = to_host(t)
    if t.dtype == torch.bfloat16:
        assert np.all(np.abs(h - v) <= np.abs(v) * 2.0 ** -8 * (1 + 1e-3) + 1e-30), what
    else:
        assert rel_l2(h, v) <= 1e-6, f"{what}: {rel_l2(h, v):.3e}"


def check_f8(y8, scale, y, block, what):
    rows, D = y.shape
    blk = block or D
    nb = -(-D // blk)
    sc = to_host(scale)
    assert sc.shape == (rows, nb)
    for j in range(nb):
        part = y[:, j * blk:(j + 1) * blk]
        s = np.maximum(np.abs(part).max(-1), 1e-30) / 448.0
        np.testing.assert_allclose(sc[:, j], s, rtol=1e-6, err_msg=what)
        q = part / s[:, None]
        got = to_host(y8[:, j * blk:(j + 1) * blk])
        step = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(np.abs(q), 1e-300))), -6, 8) - 3)
        assert np.all(np.abs(got - q) <= 0.5 * step + 1e-5 * np.maximum(np.abs(q), step)), what
        assert np.mean(got != ref.e4m3_nearest(q)) <= 1e-4 + 2.0 / q.size, what     # all but a few at the very middle


TYPES = [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None), ("f32", None)]


@pytest.mark.parametrize("io,res", TYPES)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (2, 64), (5, 100), (4, 768), (7, 2560), (3, 5120), (2, 8191), (2, 16384), (600, 520)])
def test_types_and_sizes(io, res, rows, D):
    x, r, w = inputs(rows, D, io, res)
    y, ro = ss.ss_add_rmsnorm(x, w, residual=r)
    vy, vr = want(x, r, w)
    close(y, vy, "y")
    close(ro, vr, "residual")
    for block in (0, 32, 64, 128, 256):
        y8, ro8, sc = ss.ss_add_rmsnorm_f8(x, w, residual=r, block=block)
        check_f8(y8, sc, vy, block, f"block {block}")
        assert torch.equal(ro8, ro)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("io,res", TYPES[:4])
def test_strides_and_in_place_residual(io, res, pad):
    x, r, w = inputs(9, 256, io, res, pad=pad)
    vy, vr = want(x, r, w)
    keep = r.clone()
    y, ro = ss.ss_add_rmsnorm(x, w, residual=r, residual_out=r)
    assert ro is r
    close(y, vy, "y")
    close(r, vr, "residual in place")
    wide = torch.zeros(9, 300, dtype=torch.float8_e4m3fn, device="cuda")
    y8, _, sc = ss.ss_add_rmsnorm_f8(x, w, residual=keep, block=64, y=wide[:, 3:259])
    check_f8(y8, sc, vy, 64, "strided codes")
    assert not wide[:, :3].float().any() and not wide[:, 259:].float().any()


def test_zero_rows_empty_calls_and_non_finite_rows():
    x = torch.zeros(4, 192, device="cuda")
    w = torch.ones(192, device="cuda")
    x[1, 5], x[2, 100] = float("nan"), float("inf")
    x[3, :64] = 1e-22
    y, ro = ss.ss_add_rmsnorm(x, w)
    assert not y[0].any() and torch.isnan(y[1]).all() and torch.isnan(y[2, 100]) and not y[2, :100].any()
    y8, _, sc = ss.ss_add_rmsnorm_f8(x, w, block=64)
    v = y8.float()
    assert not v[0].any() and torch.allclose(sc[0], torch.full((3,), 1e-30 / 448, device="cuda"), rtol=1e-6)
    assert torch.isnan(v[1]).all() and torch.isnan(sc[1]).all()
    assert torch.isnan(sc[2, 1]) and torch.isnan(v[2, 64:128]).all() and not v[2, :64].any()
    assert torch.isfinite(v[3]).all() and (v[3, :64] == 448).all()
    e = torch.empty(0, 192, device="cuda")
    y, ro = ss.ss_add_rmsnorm(e, w)
    assert y.shape == (0, 192)
    y8, ro, sc = ss.ss_add_rmsnorm_f8(e, w, block=128)
    assert sc.shape == (0, 2)


def test_rows_past_32_bit_offsets():
    rows, D = 300000, 8192                                   # 2.4e9 elements
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(D, device="cuda").to(torch.bfloat16)
    w = torch.ones(D, device="cuda")
    y8, ro, sc = ss.ss_add_rmsnorm_f8(x, w)
    vy, _ = ref.norm(to_host(x[-1:]), None, to_host(w), 1e-5)
    check_f8(y8[-1:], sc[-1:], vy, 0, "last row")
    assert torch.equal(ro[-1], x[-1]) and not y8[:-1:1000].float().any()


def test_refusals():
    x, r, w = inputs(4, 64, "bf16", "f32")
    with pytest.raises(ss.SelscanError):
        ss.ss_add_rmsnorm_f8(x, w, residual=r, block=48)
    with pytest.raises(ss.SelscanError):
        ss.ss_add_rmsnorm(x, w, residual=r, y=x)
    with pytest.raises(ss.SelscanError):
        ss.ss_add_rmsnorm(torch.zeros(1, 16385, device="cuda"), torch.ones(16385, device="cuda"))
    with pytest.raises(TypeError):
        ss.ss_add_rmsnorm(x.half(), w)
    with pytest.raises(ValueError):
        ss.ss_add_rmsnorm(x, w[:63])
    with pytest.raises(ValueError):
        ss.ss_add_rmsnorm(x, w, residual=r[:3])
    with pytest.raises(ValueError):
        ss.ss_add_rmsnorm(x.t(), w)
