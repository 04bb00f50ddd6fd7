"""The binding without a device."""
import inspect
import re

import torch

from bit_quantization_b200 import ops


def test_private_names_of_torch():
    """One, which this torch has; everything else is public."""
    used = set(re.findall(r"torch\._\w+(?:\.\w+)*", inspect.getsource(ops)))
    assert used == {"torch._C._cuda_getCurrentRawStream"}
    assert callable(torch._C._cuda_getCurrentRawStream)
