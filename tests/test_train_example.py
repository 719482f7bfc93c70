"""examples/train_mlp.py's arguments: sizes of nothing are refused before a GPU is asked for."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("option", ["--dim", "--hidden", "--layers", "--tokens", "--steps"])
@pytest.mark.parametrize("value", ["0", "-3"])
def test_sizes_of_nothing_are_refused(option, value, capsys):
    spec = importlib.util.spec_from_file_location("train_mlp", os.path.join(ROOT, "examples", "train_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    with pytest.raises(SystemExit) as e:
        m.main([option, value])
    assert e.value.code == 2 and f"{option} must be at least 1" in capsys.readouterr().err
