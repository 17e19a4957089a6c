"""The training example: its gradients are those of the whole model's definition in 64 bits, and it runs."""
import importlib.util
import os

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_stack.py")


@pytest.fixture
def train():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_stack", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    yield m
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def definition(model, tokens, targets, teacher, weight, temperature):
    """Loss and gradients by automatic differentiation of the model's formulas in doubles."""
    F = torch.nn.functional
    leaves = [{k: v.double().requires_grad_() for k, v in layer.p.items()} for layer in model.layers]
    own = {k: v.double().requires_grad_() for k, v in model.p.items()}
    batch, L = tokens.shape
    x = own["table"][tokens.reshape(-1).long()]
    r = torch.zeros_like(x)
    for layer, p in zip(model.layers, leaves):
        Dm, N, R = layer.Dm, layer.N, layer.R
        r = x + r
        h = F.layer_norm(r, r.shape[1:], p["norm_w"], p["norm_b"], 1e-5)
        uz = (h @ p["w_in"].t()).view(batch, L, 2 * Dm)
        v, z = uz[..., :Dm].transpose(1, 2), uz[..., Dm:]
        u = F.silu(F.conv1d(F.pad(v, (3, 0)), p["conv_w"][:, None], p["conv_b"], groups=Dm)).transpose(1, 2)
        low, B, C = (u @ p["w_x"].t()).split([R, N, N], -1)
        delta = F.softplus(low @ p["w_dt"].t() + p["dt_bias"])
        state, ys = torch.zeros(batch, Dm, N, dtype=torch.float64, device="cuda"), []
        for t in range(L):
            d = delta[:, t, :, None]
            state = torch.exp(-d * torch.exp(p["A_log"])) * state + d * u[:, t, :, None] * B[:, t, None]
            ys.append((state * C[:, t, None]).sum(-1))
        y = (torch.stack(ys, 1) + p["D"] * u) * F.silu(z)
        x = y.reshape(batch * L, Dm) @ p["w_out"].t()
    r = x + r
    h = F.layer_norm(r, r.shape[1:], own["norm_w"], own["norm_b"], 1e-5)
    logits = h @ own["head"].t()
    t = targets.reshape(-1).long()
    total = F.cross_entropy(logits, t, ignore_index=-1, reduction="sum") / (t >= 0).sum()
    if teacher is not None:
        ids, top = teacher
        lp = torch.log_softmax(top.double() / temperature, 1)
        lq = torch.gather(torch.log_softmax(logits / temperature, 1), 1, ids.long())
        total = (1 - weight) * total + weight * (lp.exp() * (lp - lq)).sum() / (batch * L)
    everything = [(i, k) for i, p in enumerate(leaves + [own]) for k in p]
    grads = torch.autograd.grad(total, [(leaves + [own])[i][k] for i, k in everything])
    return float(total.detach()), {ik: g for ik, g in zip(everything, grads)}


@pytest.mark.parametrize("distilled", [False, True])
def test_gradients_are_the_definitions(train, distilled):
    """float32: relative L2 1e-4, as the scan's own gradients are held to (two layers of it behind each other)."""
    model = train.Model(seed=2)
    g = torch.Generator("cuda").manual_seed(3)
    tokens = torch.randint(0, 500, (3, 70), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(-1, 500, (3, 70), generator=g, device="cuda", dtype=torch.int32)
    targets[:, :9] = -1
    teacher = None
    if distilled:
        top = torch.topk(3 * torch.randn(210, 500, generator=g, device="cuda"), 12)
        teacher = (top.indices.to(torch.int32), top.values)
    loss, grads = model.step(tokens, targets, teacher)
    want_loss, want = definition(model, tokens, targets, teacher, 0.5, 2.0)
    assert abs(float(loss) - want_loss) <= 1e-5 * abs(want_loss)
    assert {(i, k) for i, p in enumerate(grads) for k in p} == set(want)
    for (i, k), v in want.items():
        e = float((grads[i][k].double() - v).norm() / v.norm())
        assert e <= 1e-4, f"{i} {k}: {e:.2e}"


def test_bfloat16_step_is_near_the_float32_one(train):
    """The same step with bf16 projections and activations: gradients within some 30 roundings of 2^-9 along the
    way (each tensor's largest relative distance, by norm)."""
    a, b = train.Model(seed=4), train.Model(seed=4, dtype=torch.bfloat16)
    for la, lb in zip(a.layers, b.layers):
        la.p = {k: v.float() for k, v in lb.p.items()}
    a.p = {k: v.float() for k, v in b.p.items()}
    g = torch.Generator("cuda").manual_seed(5)
    tokens = torch.randint(0, 500, (2, 64), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(0, 500, (2, 64), generator=g, device="cuda", dtype=torch.int32)
    (la, ga), (lb, gb) = a.step(tokens, targets), b.step(tokens, targets)
    assert abs(float(la) - float(lb)) <= 0.05
    for p, q in zip(ga, gb):
        for k in p:
            assert float((p[k] - q[k].float()).norm()) <= 30 * 2.0 ** -9 * float(p[k].norm()) + 1e-6, k


def test_runs(train):
    train.main()
