"""What examples/verify_loop.py makes before it touches a device."""
import importlib.util
import os
import sys

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "verify_loop.py")
spec = importlib.util.spec_from_file_location("verify_loop", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


class Made(Exception):
    pass


@pytest.mark.parametrize("steps", [1, 32, 194, 195, 400, 5000])
def test_positions_and_pages_for_all_steps(monkeypatch, steps):
    """A step commits up to gamma + 1 = 5 tokens and writes up to 5 positions past
    what is committed; four prompts of up to 50 tokens share the pool evenly."""
    def target(page=16, pages=512, longest=1024, **kw):
        raise Made(page, pages, longest)
    monkeypatch.setattr(example, "Target", target)
    monkeypatch.setattr(sys, "argv", ["verify_loop.py", "--steps", str(steps)])
    with pytest.raises(Made) as made:
        example.main()
    page, pages, longest = made.value.args
    need = 50 + 5 * steps
    assert longest >= need and pages // 4 * page >= need
    if need <= 1024:
        assert (pages, longest) == (512, 1024)
