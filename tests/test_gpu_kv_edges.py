"""The cache's calls at the edges of what they take: states only the device knows, and values at the ends of their types.
Oracle and bounds are those of test_gpu_kv unless a test says otherwise."""

import numpy as np
import pytest

import oracle

from gpu_util import announce
from test_gpu_kv import DT, EPS, Rig, _f64, _ids

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
