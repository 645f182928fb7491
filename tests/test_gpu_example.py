"""The attention block example runs and agrees with plain torch at every stage (needs a GB300)."""
import os
import sys

import pytest

from tests.conftest import ROOT


@pytest.mark.gpu
def test_attention_block_example(capsys):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import attention_block
    finally:
        sys.path.pop(0)
    attention_block.main()
    assert capsys.readouterr().out.count("relative difference") == 9
