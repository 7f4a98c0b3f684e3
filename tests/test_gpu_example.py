"""The command line of examples/decoder_block.py: what it builds."""
import importlib.util
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")
_spec = importlib.util.spec_from_file_location("decoder_block_line", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("args,turned", [([], True), (["--projections", "torch", "--base", "0"], False),
                                         (["--base", "500000", "--cache", "bf16"], True)])
def test_command_line(monkeypatch, capsys, args, turned):
    """With the rotation and without: the block as it was before it had one."""
    made = []

    class Block(example.DecoderBlock):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            made.append(self)

    monkeypatch.setattr(example, "DecoderBlock", Block)
    monkeypatch.setattr(sys, "argv", ["decoder_block.py", "--steps", "2"] + args)
    example.main()
    assert "2 steps of 8 sequences" in capsys.readouterr().out
    assert len(made) == 1 and (made[0].rope is not None) == turned
