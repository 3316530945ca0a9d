"""The README's examples run as they stand, one after another."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_examples_run():
    from bayesian_scan_gb300 import kdn
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"^```python\n(.*?)^```", f.read(), re.M | re.S)
    assert len(blocks) >= 3
    names = {}
    for block in blocks:
        exec(compile(block, README, "exec"), names)          # noqa: S102 (the repository's own text)
    torch.cuda.synchronize()
    assert kdn.get_device_error() == kdn.KDN_OK
    assert names["o1"].shape == (1, 16, 128) and names["o1"].isfinite().all()
