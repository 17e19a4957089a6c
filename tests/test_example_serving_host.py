"""The serving example refuses prompts that it cannot take, before anything touches a device: an empty one has
no last row to draw from (it would take the one before it), and every prompt needs a slot."""
import importlib.util
import os
from types import SimpleNamespace

import pytest

pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_stack.py")


@pytest.mark.parametrize("prompts", [[], [[]], [[1, 2], []], [[], [3]], [[1]] * 5])
def test_prompts_that_are_refused(prompts):
    spec = importlib.util.spec_from_file_location("serve_stack", PATH)
    serve = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(serve)
    with pytest.raises(ValueError):
        serve.Stack.generate(SimpleNamespace(slots=4), prompts, 2)
