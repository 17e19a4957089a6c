"""Parity of the multi-head scan with its convolution (prompts and single tokens) with the 64-bit
definition.  Tolerances are the scan's own: relative L2 1e-5 for float32 outputs and states, 5e-3 for
bfloat16 outputs (their rounding, 1.7e-3, and that of operands of matrix products, each as large)."""
import ctypes

import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref
from selective_state_space_scan_gb300 import serving

from helpers import BF16_REL_L2, FP32_REL_L2, STATE_REL_L2, rel_l2, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


class Case:
    """Inputs on the device, in the layout of one projection's output when `wide`."""

    def __init__(self, lens, H=4, P=64, G=1, N=128, io="bf16", seed=0, wide=True, gate=True, bias=True, D=True, pool=None,
                 pad=0, scale=1.0, dt_shift=-4.0):
        g = torch.Generator("cuda").manual_seed(1000 + seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
        self.dt = torch.bfloat16 if io == "bf16" else torch.float32
        self.io, self.H, self.P, self.G, self.N, self.lens = io, H, P, G, N, list(lens)
        C = self.C = H * P + 2 * G * N
        T, n = sum(lens), len(lens)
        pool = n + 2 if pool is None else pool
        if wide:
            w = torch.full((T, H * P + C + H + pad), float("nan"), dtype=self.dt, device="cuda")
            z, xbc, dtr = w[:, :H * P], w[:, H * P:H * P + C], w[:, H * P + C:H * P + C + H]
        else:
            z, xbc, dtr = (torch.empty(T, k, dtype=self.dt, device="cuda") for k in (H * P, C, H))
        z.copy_(rn(T, H * P))
        xbc.copy_(scale * rn(T, C))
        dtr.copy_(rn(T, H) + dt_shift)
        self.z = z if gate else None
        self.xbc, self.dt_raw = xbc, dtr
        self.conv_w, self.conv_b = 0.5 * rn(C, 4), 0.1 * rn(C) if bias else None
        self.dt_bias = -torch.rand(H, generator=g, device="cuda") if bias else None
        self.A_log = torch.log(1 + 15 * torch.rand(H, generator=g, device="cuda"))
        self.D = 1 + 0.1 * rn(H) if D else None
        self.state, self.window = 0.5 * rn(pool, H, P, N), rn(pool, C, 3)
        self.slots = torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.lens)]), dtype=torch.int32, device="cuda")
        self.fresh = None

    def clone_caches(self):
        return self.state.clone(), self.window.clone()

    def fwd(self, state, window, **kw):
        a = dict(conv_b=self.conv_b, dt_bias=self.dt_bias, D=self.D, z=self.z, slots=self.slots, fresh=self.fresh)
        a.update(kw)
        return ss.ss_heads_fwd(self.xbc, self.dt_raw, self.conv_w, self.A_log, state, window, self.cu, **a)

    def step(self, state, window, **kw):
        a = dict(conv_b=self.conv_b, dt_bias=self.dt_bias, D=self.D, z=self.z, slots=self.slots)
        a.update(kw)
        return ss.ss_heads_step(state, window, self.xbc, self.dt_raw, self.conv_w, self.A_log, **a)

    def reference(self, state, window):
        """(y, state, window) in 64 bits of one call on these caches."""
        h = lambda t: None if t is None else to_host(t)               # noqa: E731
        y = np.zeros((sum(self.lens), self.H * self.P))
        S, W = h(state), h(window)
        slots = range(len(self.lens)) if self.slots is None else self.slots.tolist()
        fresh = [0] * len(self.lens) if self.fresh is None else self.fresh.tolist()
        xbc, dtr, z = h(self.xbc), h(self.dt_raw), h(self.z)
        par = [h(t) for t in (self.conv_w, self.conv_b, self.dt_bias, self.A_log, self.D)]
        at = 0
        for L, slot, f in zip(self.lens, slots, fresh):
            r = slice(at, at + L)
            warm = slot >= 0 and not f
            S0 = S[slot] if warm else np.zeros((self.H, self.P, self.N))
            W0 = W[slot] if warm else np.zeros((self.C, 3))
            y[r], S1, W1 = ref.heads(xbc[r], dtr[r], *par, None if z is None else z[r], S0, W0, self.P, self.N)
            if slot >= 0:
                S[slot], W[slot] = S1, W1
            at += L
        return y, S, W


def check(c, y, state, window, want, what=""):
    ry, rs, rw = want
    tol = BF16_REL_L2 if c.io == "bf16" else FP32_REL_L2
    yh, sh = to_host(y), to_host(state)
    assert np.all(np.isfinite(yh)) and np.all(np.isfinite(sh)), what
    if yh.size:
        assert rel_l2(yh, ry) <= tol, f"{what}: y rel-L2 {rel_l2(yh, ry):.3e}"
    assert rel_l2(sh, rs) <= STATE_REL_L2, f"{what}: state rel-L2 {rel_l2(sh, rs):.3e}"
    # every slot for itself: a wrong one does not hide behind the others
    for i in range(sh.shape[0]):
        assert rel_l2(sh[i], rs[i]) <= STATE_REL_L2, f"{what}: slot {i} rel-L2 {rel_l2(sh[i], rs[i]):.3e}"
    np.testing.assert_array_equal(to_host(window), rw.astype(np.float32).astype(np.float64))


def run_fwd(c, what="", **kw):
    state, window = c.clone_caches()
    want = c.reference(state, window)
    y = c.fwd(state, window, **kw)
    torch.cuda.synchronize()
    check(c, y, state, window, want, what)
    return y, state, window


IOS = ["bf16", "f32"]


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("L", [1, 2, 3, 4, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 300])
def test_lengths(io, L):
    run_fwd(Case([L], io=io, seed=L), f"L={L} {io}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("lens", [[0], [0, 0, 5], [70, 0, 1, 200, 3, 129], [1] * 9, [128, 128, 64], [511, 2, 0, 190]])
def test_packed_lengths(io, lens):
    run_fwd(Case(lens, io=io, seed=len(lens)), f"{lens} {io}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("H,P,G,N", [(1, 1, 1, 1), (3, 20, 1, 7), (2, 64, 2, 64), (6, 32, 3, 16), (5, 64, 5, 128), (2, 128, 1, 128),
                                     (2, 48, 1, 96), (1, 256, 1, 256), (4, 16, 2, 33), (8, 64, 2, 128), (3, 64, 1, 64),
                                     (2, 128, 2, 64), (4, 32, 1, 128), (7, 64, 1, 128)])
def test_shapes(io, H, P, G, N):
    run_fwd(Case([150, 37], H=H, P=P, G=G, N=N, io=io, seed=H * P + N), f"{(H, P, G, N)} {io}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("layout", ["wide", "dense", "odd", "offset"])
def test_layouts(io, layout):
    """Columns of one projection (rows on 16 bytes or not), tensors of their own, a misaligned base."""
    c = Case([140, 61], H=4, io=io, wide=layout in ("wide", "odd"), pad={"odd": 1}.get(layout, 0), seed=5)
    if layout == "offset":
        for k in ("xbc", "dt_raw", "z"):
            t = getattr(c, k)
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view_as(t)
            flat.copy_(t)
            setattr(c, k, flat)
    run_fwd(c, f"{layout} {io}")
    buf = torch.full((201, c.H * c.P + 9), float("nan"), dtype=c.dt, device="cuda")
    y = buf[:, 1:1 + c.H * c.P]                          # y in a wider buffer, off its alignment
    run_fwd(c, f"{layout} {io} strided y", y=y)
    assert torch.isnan(buf[:, 0]).all() and torch.isnan(buf[:, 1 + c.H * c.P:]).all()


@pytest.mark.parametrize("opt", ["gate", "bias", "D"])
@pytest.mark.parametrize("io", IOS)
def test_optional_inputs(io, opt):
    run_fwd(Case([133, 20], io=io, seed=3, **{opt: False}), f"no {opt} {io}")


@pytest.mark.parametrize("io", IOS)
def test_fresh_and_slotless_sequences(io):
    """A fresh sequence reads nothing of its slot (NaN there stays out of it); one without a slot starts
    from zeros and leaves nothing; the default slots are the sequences' own numbers."""
    c = Case([130, 40, 0, 200, 0], io=io, seed=11, pool=7)
    c.slots = torch.tensor([4, -1, 2, 0, 6], dtype=torch.int32, device="cuda")
    c.fresh = torch.tensor([1, 0, 1, 0, 0], dtype=torch.int32, device="cuda")
    state, window = c.clone_caches()
    want = c.reference(state, window)
    for k in (4, 2):
        state[k], window[k] = float("nan"), float("nan")
    y = c.fwd(state, window)
    torch.cuda.synchronize()
    check(c, y, state, window, want)
    assert (state[2] == 0).all() and (window[2] == 0).all()        # empty and fresh: zeros
    c.slots, c.fresh = None, None
    run_fwd(c, "default slots")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("cut", [1, 2, 3, 64, 128, 131])
def test_prompt_in_two_calls(io, cut):
    """A prompt in two calls on the same slot leaves what one call leaves."""
    c = Case([300], io=io, seed=cut)
    y, state, window = run_fwd(c)
    s2, w2 = c.clone_caches()
    parts = []
    for a, b in ((0, cut), (cut, 300)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        parts.append(ss.ss_heads_fwd(c.xbc[a:b], c.dt_raw[a:b], c.conv_w, c.A_log, s2, w2, cu, conv_b=c.conv_b,
                                     dt_bias=c.dt_bias, D=c.D, z=c.z[a:b], slots=c.slots))
    torch.cuda.synchronize()
    tol = 2 * (BF16_REL_L2 if io == "bf16" else FP32_REL_L2)
    assert rel_l2(to_host(torch.cat(parts)), to_host(y)) <= tol
    assert rel_l2(to_host(s2), to_host(state)) <= 2 * STATE_REL_L2
    assert torch.equal(w2, window)


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("H,P,G,N", [(1, 1, 1, 1), (3, 20, 1, 7), (2, 64, 2, 64), (6, 32, 3, 16), (5, 64, 5, 128), (2, 128, 1, 32),
                                     (2, 48, 1, 96), (1, 256, 1, 256), (24, 64, 1, 128), (4, 72, 2, 64)])
def test_step_shapes(io, H, P, G, N):
    for batch in (1, 5):
        c = Case([1] * batch, H=H, P=P, G=G, N=N, io=io, seed=H + N + batch)
        state, window = c.clone_caches()
        for k in range(3):                                  # three tokens on the same caches
            want = c.reference(state, window)
            y = c.step(state, window)
            torch.cuda.synchronize()
            check(c, y, state, window, want, f"step {k} {(H, P, G, N)} {io}")


@pytest.mark.parametrize("io", IOS)
def test_step_padded_rows_and_layouts(io):
    c = Case([1] * 6, io=io, seed=21, pool=9, pad=1)
    c.slots = torch.tensor([3, -1, 8, 0, -5, 1], dtype=torch.int32, device="cuda")
    state, window = c.clone_caches()
    want = c.reference(state, window)
    y = c.step(state, window)
    torch.cuda.synchronize()
    check(c, y, state, window, want)
    c.slots = None
    state, window = c.clone_caches()
    want = c.reference(state, window)
    y = c.step(state, window)
    check(c, y, state, window, want)


@pytest.mark.parametrize("io", IOS)
def test_steps_continue_a_prompt(io):
    """Prompt, then tokens one by one, against one long prompt."""
    c = Case([140], io=io, seed=8)
    y, state, window = run_fwd(c)
    s2, w2 = c.clone_caches()
    cu = torch.tensor([0, 130], dtype=torch.int32, device="cuda")
    kw = dict(conv_b=c.conv_b, dt_bias=c.dt_bias, D=c.D, slots=c.slots)
    ss.ss_heads_fwd(c.xbc[:130], c.dt_raw[:130], c.conv_w, c.A_log, s2, w2, cu, z=c.z[:130], **kw)
    ys = [ss.ss_heads_step(s2, w2, c.xbc[t:t + 1], c.dt_raw[t:t + 1], c.conv_w, c.A_log, z=c.z[t:t + 1], **kw)
          for t in range(130, 140)]
    torch.cuda.synchronize()
    tol = 2 * (BF16_REL_L2 if io == "bf16" else FP32_REL_L2)
    assert rel_l2(to_host(torch.cat(ys)), to_host(y[130:])) <= tol
    assert rel_l2(to_host(s2), to_host(state)) <= 2 * STATE_REL_L2
    assert torch.equal(w2, window)


def test_strong_and_weak_decay():
    """Time steps from 1e-4 to 10 and more: decays that vanish within a step, and states that hardly do."""
    for shift, seed in ((-9.0, 1), (0.0, 2), (6.0, 3)):
        for io in IOS:
            run_fwd(Case([200, 131], io=io, seed=seed, dt_shift=shift), f"shift {shift} {io}")


def test_state_offsets_past_32_bits():
    """A pool of more than 2^31 state values: the last slots are reached by both calls."""
    H, P, N, pool = 64, 64, 128, 4104
    c = Case([17, 33], H=H, P=P, N=N, seed=4, pool=2)
    small_s, small_w = c.clone_caches()
    c.slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want = c.reference(small_s, small_w)
    state = torch.zeros(pool, H, P, N, device="cuda")
    window = torch.zeros(pool, c.C, 3, device="cuda")
    state[-2:], window[-2:] = small_s, small_w
    c.slots = torch.tensor([pool - 2, pool - 1], dtype=torch.int32, device="cuda")
    y = c.fwd(state, window)
    torch.cuda.synchronize()
    check(c, y, state[-2:], window[-2:], want)
    assert not state[:-2].any()
    d = Case([1, 1], H=H, P=P, N=N, seed=4, pool=2)
    d.slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    s0, w0 = state[-2:].clone(), window[-2:].clone()
    want = d.reference(s0, w0)
    d.slots = c.slots
    y = d.step(state, window)
    torch.cuda.synchronize()
    check(d, y, state[-2:], window[-2:], want)
    assert not state[:-2].any()


def test_side_stream_and_repeats_are_bitwise_equal():
    c = Case([257, 0, 90], H=6, seed=31)
    s0, w0 = c.clone_caches()
    y0 = c.fwd(s0, w0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s1, w1 = c.clone_caches()
    side.wait_stream(torch.cuda.current_stream())
    y1 = c.fwd(s1, w1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(s0, s1) and torch.equal(w0, w1)


def test_indexes_out_of_range_are_reported_and_skipped():
    c = Case([40, 50], seed=6, pool=2)
    state, window = c.clone_caches()
    c.slots = torch.tensor([5, 1], dtype=torch.int32, device="cuda")
    y = torch.full((90, c.H * c.P), 7.0, dtype=c.dt, device="cuda")
    c.fwd(state, window, y=y)
    assert ss.device_error(clear=True) == 4
    assert (y[:40] == 7).all() and torch.equal(state[0], c.state[0])
    c.slots = None
    state, window = c.clone_caches()
    c.cu = torch.tensor([0, 40, 91], dtype=torch.int32, device="cuda")       # one row too many
    y = torch.full((90, c.H * c.P), 7.0, dtype=c.dt, device="cuda")
    c.fwd(state, window, y=y)
    assert ss.device_error(clear=True) == 4
    assert (y[40:] == 7).all() and not (y[:40] == 7).all() and torch.equal(state[1], c.state[1])
    c.cu = torch.tensor([0, -3, 20], dtype=torch.int32, device="cuda")
    c.fwd(state, window, y=y)
    assert ss.device_error(clear=True) == 4
    d = Case([1, 1], seed=6, pool=2)
    d.slots = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    state, window = d.clone_caches()
    y = torch.full((2, d.H * d.P), 7.0, dtype=d.dt, device="cuda")
    d.step(state, window, y=y)
    assert ss.device_error(clear=True) == 4
    assert (y[1] == 7).all() and torch.equal(state[0], d.state[0]) and not torch.equal(state[1], d.state[1])


def test_overlaps_are_refused():
    c = Case([40], seed=7)
    state, window = c.clone_caches()
    with pytest.raises(ss.SelscanError):
        c.fwd(state, window, y=c.z)                                         # y over z
    with pytest.raises(ss.SelscanError):
        c.fwd(state, state.view(-1)[:window.numel()].view_as(window))        # window inside state


class Force:
    """Takes the library's choice of path and of segments out of its hands for a while."""

    def __init__(self, path=0, chunks=0, pre=0):
        self.path, self.chunks, self.pre = path, chunks, pre

    def __enter__(self):
        lib = ss.lib()
        for f in (lib.ss__force_heads_path, lib.ss__force_heads_chunks, lib.ss__force_heads_pre):
            f.argtypes = [ctypes.c_int]
        lib.ss__force_heads_path(self.path)
        lib.ss__force_heads_chunks(self.chunks)
        lib.ss__force_heads_pre(self.pre)
        serving._HEADS_BYTES.clear()

    def __exit__(self, *a):
        ss.lib().ss__force_heads_path(0)
        ss.lib().ss__force_heads_chunks(0)
        ss.lib().ss__force_heads_pre(0)
        serving._HEADS_BYTES.clear()


@pytest.mark.parametrize("L", [1, 2, 3, 4, 17, 31, 32, 33, 64, 96, 97, 127, 128, 129, 130, 131, 255, 257])
def test_products_at_every_length(L):
    """Chunks of every fill, from the slot's state and from zeros."""
    with Force(path=2):
        run_fwd(Case([L], H=3, seed=L), f"products L={L}")
        run_fwd(Case([5, L, 0, L + 130, 1], H=2, N=48, P=40, seed=L), f"products packed L={L}")


@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("L", [70, 256, 1000])
def test_token_by_token_at_long_lengths(io, L):
    with Force(path=1):
        run_fwd(Case([L, 3, L // 2], H=3, io=io, seed=L), f"tokens L={L} {io}")
        run_fwd(Case([L], H=1, P=64, N=200, io=io, seed=L), f"tokens L={L} N=200 {io}")


@pytest.mark.parametrize("pre", [1, 2])
@pytest.mark.parametrize("io", IOS)
@pytest.mark.parametrize("H,P,G,N", [(2, 64, 1, 128), (3, 20, 3, 7), (4, 72, 2, 64), (2, 100, 1, 32), (1, 64, 1, 16)])
def test_token_by_token_with_b_and_c_beforehand(io, pre, H, P, G, N):
    with Force(path=1, pre=pre):
        run_fwd(Case([1, 0, 15, 16, 17, 200, 33, 130, 2], H=H, P=P, G=G, N=N, io=io, seed=H + N), f"{(H, P, G, N)} {io} {pre}")
        run_fwd(Case([900], H=H, P=P, G=G, N=N, io=io, seed=N), f"long {(H, P, G, N)} {io} {pre}")


@pytest.mark.parametrize("chunks", [1, 2, 3, 7, -1, -2, -3, -100])
def test_segments_of_any_length(chunks):
    """The time split (two passes) and the waves (the state handed from CTA to CTA) at every cut, with
    sequences that end inside, at and before a segment's end, fresh ones and slotless ones."""
    lens = [700, 128, 0, 385, 256, 60, 512]
    c = Case(lens, H=5, seed=40 + abs(chunks))
    c.fresh = torch.tensor([0, 1, 0, 1, 0, 0, 0], dtype=torch.int32, device="cuda")
    c.slots[4] = -1
    with Force(path=2, chunks=chunks):
        first = run_fwd(c, f"segments of {chunks}")
        again = run_fwd(c, f"segments of {chunks}")
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_more_segments_than_ctas():
    """Waves of many more segments than the device has SMs, of sequences of unlike lengths."""
    lens = [1300, 40, 900, 640, 128, 129, 1, 500]
    with Force(path=2, chunks=-1):
        run_fwd(Case(lens, H=96, P=64, N=32, G=1, seed=50), "many segments")


@pytest.mark.parametrize("io,path", [("bf16", 2), ("bf16", 1), ("f32", 1)])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", [0, 37, 150, 255])
def test_what_is_not_finite_stays_in_its_place(io, path, what, value, at):
    """An infinite or NaN input reaches the outputs and states that the recurrence takes it to, and no
    others: not the tokens before it, the other channels or the other sequence."""
    c = Case([300, 70], H=4, P=40, N=48, io=io, seed=60 + at)
    if what == "dt":
        c.dt_raw[at, 1] = value
    else:
        first = {"x": c.P + 5, "B": c.H * c.P + 7, "C": c.H * c.P + c.N + 7}[what]
        c.xbc[at, first] = value
    state, window = c.clone_caches()
    with np.errstate(invalid="ignore", over="ignore"):
        ry, rs, rw = c.reference(state, window)
    with Force(path=path):
        y = to_host(c.fwd(state, window))
    sh = to_host(state)
    for got, want, tol in ((y, ry, BF16_REL_L2 if io == "bf16" else FP32_REL_L2), (sh, rs, STATE_REL_L2)):
        on = np.isfinite(want)
        np.testing.assert_array_equal(np.isfinite(got), on)
        assert rel_l2(got[on], want[on]) <= tol
    np.testing.assert_array_equal(to_host(window), rw.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("pad", [0, 1, 2])
@pytest.mark.parametrize("H,P,G,N", [(3, 20, 1, 7), (1, 1, 1, 1), (5, 37, 5, 33), (4, 63, 2, 128), (2, 127, 1, 61), (3, 66, 1, 16)])
def test_products_at_any_alignment(H, P, G, N, pad):
    """Rows of the products' path that begin anywhere, tiles that end anywhere; what lies between the rows
    is NaN."""
    c = Case([150, 37, 0, 129], H=H, P=P, G=G, N=N, pad=pad, seed=70 + pad)
    wide = torch.full((316, c.C + 2 + pad), float("nan"), dtype=c.dt, device="cuda")
    gate = torch.full((316, H * P + 1 + 2 * pad), float("nan"), dtype=c.dt, device="cuda")
    wide[:, 1:1 + c.C], gate[:, :H * P] = c.xbc, c.z
    out = torch.full((316, H * P + 2 + pad), float("nan"), dtype=c.dt, device="cuda")
    with Force(path=2):
        run_fwd(c, f"{(H, P, G, N)} pad {pad}")
        c.xbc, c.z = wide[:, 1:1 + c.C], gate[:, :H * P]
        run_fwd(c, f"{(H, P, G, N)} pad {pad}, apart", y=out[:, 1:1 + H * P])
    assert torch.isnan(out[:, 0]).all() and torch.isnan(out[:, 1 + H * P:]).all()
