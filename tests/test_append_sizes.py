"""rotate_append's launch arithmetic at the largest token counts, on the host: without a GPU the launch
itself fails (status 4), which is what shows that the sizes before it came out."""
import subprocess
import sys

import pytest
import torch

import sparse_moe_layer_gb300 as moe

CALL = """
import struct, sparse_moe_layer_gb300 as moe
kv = struct.Struct("4P9q5i4x").pack(256, 512, 0, 0, *([2048, 1024, 64] * 2), 32, 16, 1, 0, 4, 16, 2, 64)
for n in (2 ** 31 - 1, 2 ** 31 - 7, 2 ** 31 - 8, 2 ** 31 - 1300, 2 ** 30, 3, 1):
    s = moe.lib().moe_rotate_append(kv, 256, 256, 256, 0, 0, 64, 0, 64, 0, 64, 256, 256, 256, 64, 0, 1.0, n, 4, 256, 256, 64,
                                    None, None)
    assert s == 4, (n, s)
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: nothing may be launched")
def test_token_counts_up_to_31_bits():
    moe.build()
    r = subprocess.run([sys.executable, "-c", CALL], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
