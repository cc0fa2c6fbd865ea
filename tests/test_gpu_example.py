"""The format comparison example on a small layer: the operators together, as
they are used; needs an MI355X."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_compare_formats(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import compare_formats

    rows = {r[0]: r[1:] for r in compare_formats.main(["--tokens", "200", "--d-in", "1024", "--d", "256", "--vocab", "3000"])}
    assert "gradient cosine" in capsys.readouterr().out
    assert set(rows) == {"bf16", "qamw", "mxfp4", "mxfp4+rot"}
    for name, (layer, out, loss, change, cos) in rows.items():
        # 4-bit weights alone are within 15 %, weights and activations within 25 %, of the layer's output
        assert layer < 0.15 and out < 0.25 and abs(change) < 0.2 and cos > 0.9, name
    # the rotation spreads the outlier channels that the plain format spends its scales on
    assert rows["mxfp4+rot"][1] < rows["mxfp4"][1]
