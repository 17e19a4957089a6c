"""The serving example: packed prompts and tokens one by one give what one packed call gives, and a
conversation's tokens do not depend on its neighbours."""
import importlib.util
import os

import pytest

import selective_state_space_scan_gb300 as ss

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_stack.py")


@pytest.fixture
def serve():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("serve_stack", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    yield m
    torch.cuda.synchronize()
    assert ss.device_error(clear=True) == 0


def test_prompt_then_tokens_equal_one_call(serve):
    """Teacher forcing: logits of the last rows from one packed call, and token by token after a prefix.
    The layers' bfloat16 activations differ by their rounding (the two paths round C·S and P·x apart)."""
    stack = serve.Stack(seed=3)
    t = torch.randint(0, 1000, (200,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    fresh = torch.ones(1, dtype=torch.int32, device="cuda")
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")             # noqa: E731
    whole = stack(t, slots, cu(200), fresh)[190:].float()
    stack(t[:190], slots, cu(190), fresh)
    steps = torch.cat([stack(t[i:i + 1], slots) for i in range(190, 200)]).float()
    assert float((steps - whole).norm() / whole.norm()) <= 3e-2
    assert float((steps.argmax(1) == whole.argmax(1)).float().mean()) >= 0.8


def test_greedy_tokens_do_not_depend_on_the_batch(serve):
    prompts = [list(range(5, 305)), [7, 8, 9], list(range(100, 160))]
    together = serve.Stack(seed=4).generate(prompts, 6, temperature=0.0)
    alone = torch.cat([serve.Stack(seed=4).generate([p], 6, temperature=0.0) for p in prompts])
    # (a near tie may fall the other way where another number of rows changes a projection's rounding)
    assert float((together == alone).float().mean()) >= 0.8
    assert torch.equal(together[:, 0], alone[:, 0]) or float((together == alone).float().mean()) >= 0.9


def test_generate_is_reproducible(serve):
    prompts = [[1, 2, 3, 4], list(range(40, 240))]
    a = serve.Stack(seed=5).generate(prompts, 8, seed=9)
    b = serve.Stack(seed=5).generate(prompts, 8, seed=9)
    assert torch.equal(a, b) and int(a.min()) >= 0 and int(a.max()) < 1000
