"""smoke() runs every family of operators."""
import pytest

import __graft_entry__ as entry

pytestmark = pytest.mark.gpu


def test_smoke_runs_the_scan_and_the_layer_operators(capsys):
    entry.smoke()
    said = capsys.readouterr().out
    assert "path=tcgen05" in said and "path=simt" in said and "layer operators" in said
