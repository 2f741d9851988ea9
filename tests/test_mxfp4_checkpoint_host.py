"""Weights that are in MXFP4 already: scales [.., rows, D / 32] into the layout of MxFp4 by the
lines that the README gives."""
import re
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")

from tests import mxfp4  # noqa: E402


@pytest.mark.parametrize("shape", [(3, 64), (2, 8, 32), (4, 40, 96), (1, 5, 1440), (2, 12, 256)])
def test_readme_lines(shape):
    import combine_moe_plan_02_gb300 as moe
    text = (Path(__file__).parent.parent / "README.md").read_text()
    lines = re.search(r"```python\n(s = torch.nn.functional.pad\(scales.*?)```", text, re.S).group(1)
    g = torch.Generator().manual_seed(shape[-1])
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(100, 140, (*shape[:-1], shape[-1] // 32), generator=g, dtype=torch.uint8)
    names = {"torch": torch, "moe": moe, "codes": codes, "scales": scales}
    exec(lines, names)
    w = names["w"]
    assert w.shape == shape and w.scales.is_contiguous()
    assert w.scales.shape == (*shape[:-2], -(-shape[-1] // 128), shape[-2], 4)
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = mxfp4.MAGNITUDES[v & 7] * (1.0 - 2.0 * (v >> 3))
    want = v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    assert torch.equal(mxfp4.values(*w), want)
    # scales past a row's end are zero, as the products ask
    assert int(w.scales.transpose(-2, -3).flatten(-2)[..., shape[-1] // 32:].sum()) == 0
