"""The sampler against the definition in 64 bits, row by row: whole numbers, so they have to be equal.
A row can differ only where the two leading tokens of the race, or a filter's edge on the winning
token, agree to about 1e-6; the inputs are fixed, and such rows are not among them."""
import numpy as np
import pytest

import selective_state_space_scan_gb300 as ss
import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.synchronize()


def noise_for(rows, V, seed=0):
    g = torch.Generator("cuda").manual_seed(77 + seed)
    return torch.empty(rows, V, device="cuda").exponential_(generator=g)


def check(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None):
    dev = lambda v, t: None if v is None else torch.tensor(v, dtype=t, device="cuda")     # noqa: E731
    got = ss.ss_sample(logits, noise, dev(temperature, torch.float32), dev(top_k, torch.int32), dev(top_p, torch.float32),
                       dev(min_p, torch.float32)).tolist()
    l, e = logits.float().cpu().numpy(), noise.cpu().numpy()
    f = lambda v, i, d: d if v is None else float(np.float32(v[i]))                       # noqa: E731
    want = [ref.sample_row(l[i], e[i], f(temperature, i, 1.0), 0 if top_k is None else top_k[i], f(top_p, i, 1.0), f(min_p, i, 0.0))
            for i in range(len(l))]
    assert got == want
    return got


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 1000, 4099, 50257, 131072])
def test_every_filter(io, V):
    g = torch.Generator("cuda").manual_seed(V)
    settings = [(1.0, 0, 1.0, 0.0), (0.0, 5, 0.5, 0.1), (0.7, 1, 1.0, 0.0), (0.9, 40, 1.0, 0.0), (1.2, 0, 0.9, 0.0),
                (0.8, 0, 0.999, 0.0), (1.0, 0, 1.0, 0.05), (0.6, 50, 0.95, 0.02), (1.0, V - 1, 0.3, 0.0), (2.0, 1500, 0.97, 0.0),
                (1.0, 0, 0.0, 0.0), (1.0, 0, -1.0, 0.0), (1.0, 3, 0.0, 2.0), (50.0, 0, 0.5, 0.0), (0.01, 0, 0.99, 0.0),
                (1.0, V + 9, 2.0, -1.0), (1.0, 20000, 0.9999, 0.0), (100.0, 30000, 0.7, 0.0)]
    rows = len(settings)
    logits = (2.5 * torch.randn(rows, V, generator=g, device="cuda")).to(DT[io])
    t, k, p, m = (list(v) for v in zip(*settings))
    for seed in range(3):
        check(logits, noise_for(rows, V, seed), t, k, p, m)
    check(logits, noise_for(rows, V, 9))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("values", [1, 2, 5])
def test_equal_logits_stay_by_index(io, values):
    """Rows of a few distinct values: every filter's edge falls among equal logits, thousands of them."""
    V = 9001
    g = torch.Generator("cuda").manual_seed(values)
    settings = [(1.0, 1, 1.0, 0.0), (1.0, 2, 1.0, 0.0), (1.0, 1025, 1.0, 0.0), (1.0, 4500, 1.0, 0.0), (1.0, 0, 0.5, 0.0),
                (1.0, 0, 0.013, 0.0), (3.0, 7000, 0.7, 0.0), (1.0, 1200, 0.001, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 8000, 0.99, 0.9)]
    rows = len(settings)
    logits = torch.randint(0, values, (rows, V), generator=g, device="cuda").to(DT[io])
    t, k, p, m = (list(v) for v in zip(*settings))
    for seed in range(4):
        check(logits, noise_for(rows, V, seed), t, k, p, m)
    same = torch.ones(rows, V, device="cuda")
    got = ss.ss_sample(logits, same).tolist()                 # a race of equals: the lowest index
    assert got == [int(torch.nonzero(r == r.max())[0]) for r in logits.float()]


def test_masked_infinite_and_empty_rows():
    V = 3001
    g = torch.Generator("cuda").manual_seed(3)
    l = torch.randn(9, V, generator=g, device="cuda")
    inf = float("inf")
    l[0] = -inf                                              # nothing left
    l[1] = float("nan")
    l[2, :] = -inf
    l[2, 1717] = -5.0                                        # one token
    l[3, 100:] = torch.finfo(torch.float32).min              # masked with the type's lowest value
    l[4, [5, 9]] = inf
    l[5, 10] = float("nan")
    l[6, :] = torch.finfo(torch.float32).min
    l[7, 1:] = -inf
    l[8, ::2] = -inf
    for k, p in ((0, 1.0), (50, 0.9), (0, 0.8), (2500, 1.0), (2500, 0.999)):
        got = check(l, noise_for(9, V, k), [0.8] * 9, [k] * 9, [p] * 9, [0.0] * 9)
        assert got[:3] == [-1, -1, 1717] and got[7] == 0 and got[4] in (5, 9) and got[5] != 10
    assert check(l, noise_for(9, V, 1), [0.0] * 9)[:2] == [-1, -1]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_row_strides_and_alignment(io):
    g = torch.Generator("cuda").manual_seed(12)
    wide = (2 * torch.randn(6, 5011, generator=g, device="cuda")).to(DT[io])
    noise = noise_for(6, 5020)[:, 3:5003]
    for off in range(4):
        check(wide[:, off:off + 5000], noise, [0.9] * 6, [0, 100, 0, 7, 0, 2000], [1.0, 0.9, 0.8, 1.0, 0.95, 0.9], [0.0] * 6)


def test_draws_follow_the_weights():
    """20000 races on one row: the tokens' frequencies are the filtered weights (4 standard deviations)."""
    n, V = 20000, 64
    logits = torch.linspace(-2, 2, V, device="cuda")[None].expand(n, V)
    got = ss.ss_sample(logits, noise_for(n, V), top_k=torch.full((n,), 10, dtype=torch.int32, device="cuda"))
    w = torch.softmax(logits[0].double(), 0)
    w[:V - 10] = 0
    w = (w / w.sum()).cpu().numpy()
    freq = np.bincount(got.cpu().numpy(), minlength=V) / n
    assert np.all(np.abs(freq - w) <= 4 * np.sqrt(w * (1 - w) / n) + 1e-12)


def test_refusals():
    l, e = torch.zeros(2, 10, device="cuda"), torch.ones(2, 10, device="cuda")
    with pytest.raises(TypeError):
        ss.ss_sample(l.half(), e)
    with pytest.raises(TypeError):
        ss.ss_sample(l, e, top_k=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError):
        ss.ss_sample(l, e[:1])
    with pytest.raises(ValueError):
        ss.ss_sample(l, e, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        ss.ss_sample(l.cpu(), e)
    with pytest.raises(ss.SelscanError):
        ss.ss_sample(torch.zeros(1, (1 << 20) + 1, device="cuda"), torch.ones(1, (1 << 20) + 1, device="cuda"))
