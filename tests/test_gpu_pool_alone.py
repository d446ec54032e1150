"""GPU: a pool's pages are created and moved with numpy alone, in a process that
has no torch to import."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys
sys.modules["torch"] = None  # any import of it fails
import numpy as np
from quantized_linear_attention_decode_b200 import stq
pool = stq.stq_pool_create(stq.STQ_GDN, 2, 2, 3, np.array([6, 4, 8], np.uint8))
assert stq.stq_pool_device(pool) == pool.device_index == 0
page = np.random.default_rng(0).integers(0, 256, pool.slot_bytes).astype(np.uint8)
stq.stq_import_slot(pool, 1, 0, page)
assert np.array_equal(stq.stq_export_slot(pool, 1, 0), page)
assert not np.array_equal(stq.stq_export_slot(pool, 0, 1), page)
pool.close()
print("done")
"""


def test_pool_without_torch():
    out = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "done", out.stderr[-2000:]


def test_device_of_a_pool():
    torch = pytest.importorskip("torch")
    import numpy as np

    from quantized_linear_attention_decode_b200 import stq
    pool = stq.stq_pool_create(stq.STQ_GDN, 1, 1, 1, np.array([6], np.uint8))
    assert pool.device == torch.device("cuda", torch.cuda.current_device())
    assert stq.stq_pool_device(pool) == torch.cuda.current_device()
