"""Parity of the convolution's backward pass with the 64-bit definition.  Tolerances: float32 relative L2 2e-6
(σ by the SFU's exponential and reciprocal, 2^-22 each, and some eight roundings of 2^-24), bfloat16 the half
step of its rounding beside that."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import training_ref as ref

from helpers import rel_l2, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2e-6


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def close(t, v, what, tol=F32):
    h = to_host(t)
    if t.dtype == torch.bfloat16:
        scale = np.sqrt(np.mean(v * v))
        assert np.all(np.abs(h - v) <= np.abs(v) * 2.0 ** -8 + 4 * tol * (np.abs(v) + scale)), what
    else:
        assert rel_l2(h, v) <= tol, f"{what}: {rel_l2(h, v):.3e}"


def case(batch, L, Dm, io="f32", pad=0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + 11 * L + Dm)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")          # noqa: E731
    x, dout = (rn(batch, L, Dm + pad).to(DT[io])[..., :Dm] for _ in range(2))
    return dict(dout=dout, x=x, weight=0.5 * rn(Dm, 4), bias=0.1 * rn(Dm), window_in=rn(batch, Dm, 3), dwindow_out=rn(batch, Dm, 3))


def check(c, silu=True):
    h = {k: None if v is None else to_host(v) for k, v in c.items()}
    dx, dw, db, dwin = ref.conv1d_bwd(h["dout"], h["x"], h["weight"], h["bias"], h["window_in"], h["dwindow_out"], silu)
    g = ss.ss_conv1d_bwd(silu=silu, **c)
    close(g["dx"], dx, "dx")
    close(g["dweight"], dw, "dweight")
    close(g["dbias"], db, "dbias")
    if c["window_in"] is None:
        assert g["dwindow_in"] is None
    else:
        close(g["dwindow_in"], dwin, "dwindow_in")
    return g


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,Dm", [(1, 1, 1), (2, 2, 5), (1, 3, 64), (3, 4, 516), (2, 45, 1536), (1, 100, 513), (2, 700, 96), (8, 33, 32),
                                        (1, 5000, 40)])
@pytest.mark.parametrize("silu", [True, False])
def test_sizes(io, batch, L, Dm, silu):
    check(case(batch, L, Dm, io), silu)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("without", ["bias", "window_in", "dwindow_out"])
def test_optional_arguments(io, without):
    c = case(2, 50, 64, io)
    c[without] = None
    check(c)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 4])
def test_strides(io, pad):
    check(case(3, 70, 64, io, pad=pad))
    c = case(3, 70, 64, io)
    c["dout"] = c["dout"][:1].expand(3, 70, 64)
    check(c)
    c["x"] = c["x"].transpose(0, 1).contiguous().transpose(0, 1)         # steps outermost
    out = torch.full((70, 3, 80), 7.0, dtype=DT[io], device="cuda").transpose(0, 1)[..., 8:72]
    g = ss.ss_conv1d_bwd(dx=out, **c)
    assert g["dx"] is out and torch.equal(out, ss.ss_conv1d_bwd(**c)["dx"])


def test_gradients_of_the_forward_call():
    """Directional differences of ss_conv1d itself, in float32: a step of 2^-6 along a random direction has a
    truncation of some 2^-12 of its second derivatives and the outputs' rounding 2^-24 · 2^6 behind it."""
    c = case(2, 40, 32)
    win = torch.empty_like(c["window_in"])

    def f(x, w, b, wi):
        out = ss.ss_conv1d(x, w, b, window_in=wi, window_out=win, silu=True)
        return float((out.double() * c["dout"]).sum() + (win.double() * c["dwindow_out"]).sum())
    g = ss.ss_conv1d_bwd(**c)
    at = [c["x"], c["weight"], c["bias"], c["window_in"]]
    for i, k in enumerate(("dx", "dweight", "dbias", "dwindow_in")):
        torch.manual_seed(i)
        d = torch.randn_like(at[i])
        step = 2.0 ** -6
        move = lambda s: f(*[a + s * d if j == i else a for j, a in enumerate(at)])          # noqa: E731
        want = float((g[k].double() * d).sum())
        size = float((g[k].double().abs() * d.abs()).sum())
        assert abs((move(step) - move(-step)) / (2 * step) - want) <= 1e-3 * size, k


def test_large_arguments():
    """v far below zero: the slope of silu is zero there, without NaN."""
    c = case(1, 9, 8)
    c["bias"] = torch.tensor([-1e4, 1e4, -90.0, 90.0, -30.0, 30.0, 0.0, -3e38], device="cuda")
    check(c)


def test_infinities_stay_in_their_channel_and_steps():
    c = case(1, 30, 8)
    c["x"][0, 10, 3] = float("inf")
    g = ss.ss_conv1d_bwd(**c)
    bad = ~torch.isfinite(g["dx"])
    assert bad[0, :, 3].any() and not bad[0, :7].any() and not bad[0, 14:].any() and not bad[..., [0, 1, 2, 4, 5, 6, 7]].any()
    assert torch.isfinite(g["dweight"][[0, 1, 2, 4, 5, 6, 7]]).all()


def test_no_steps():
    c = case(2, 0, 16)
    g = ss.ss_conv1d_bwd(**c)
    assert g["dx"].shape == (2, 0, 16) and not g["dweight"].any() and not g["dbias"].any()
    assert torch.equal(g["dwindow_in"], c["dwindow_out"])


def test_same_bits_every_time():
    c = case(4, 999, 100, "bf16")
    a, b = check(c), check(c)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_steps_past_32_bit_offsets():
    batch, L, Dm = 3, 700000, 1024                            # 2.15e9 elements
    x = torch.zeros(batch, L, Dm, dtype=torch.bfloat16, device="cuda")
    dout = torch.zeros_like(x)
    g = torch.Generator("cuda").manual_seed(1)
    x[-1, -50:] = torch.randn(50, Dm, generator=g, device="cuda").to(torch.bfloat16)
    dout[-1, -50:] = torch.randn(50, Dm, generator=g, device="cuda").to(torch.bfloat16)
    w = 0.5 * torch.randn(Dm, 4, generator=g, device="cuda")
    got = ss.ss_conv1d_bwd(dout, x, w)
    dx, dw, db, _ = ref.conv1d_bwd(to_host(dout[-1:, -60:]), to_host(x[-1:, -60:]), to_host(w), None, None, None, True)
    close(got["dx"][-1:, -60:], dx, "last steps")
    close(got["dweight"], dw, "dweight")
    close(got["dbias"], db, "dbias")
    assert not got["dx"][0, ::1000].any()


def test_refusals():
    c = case(2, 10, 16)
    with pytest.raises(ss.SelscanError):
        ss.ss_conv1d_bwd(dx=c["dout"], **c)
    with pytest.raises(ValueError):
        ss.ss_conv1d_bwd(**{**c, "dout": c["dout"][:, :9]})
    with pytest.raises(TypeError):
        ss.ss_conv1d_bwd(**{**c, "dout": c["dout"].bfloat16()})
    with pytest.raises(ValueError):
        ss.ss_conv1d_bwd(**{**c, "weight": c["weight"][:, :3]})
    with pytest.raises(ValueError):
        ss.ss_conv1d_bwd(**{**c, "window_in": c["window_in"][:1]})
