"""The example runs, with its own checks."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")


def load():
    spec = importlib.util.spec_from_file_location("decoder_layer_example", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_decoder_layer_imports():
    assert callable(load().main)


@pytest.mark.gpu
def test_decoder_layer_runs(capsys):
    load().main()
    assert "decoder layer ok" in capsys.readouterr().out
