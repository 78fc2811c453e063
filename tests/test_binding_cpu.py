"""The compiled binding and its build, without device calls."""
import subprocess
import sys

import pytest

from weight_quantized_mixed_amd import qgemm as q

CALL = """
import ctypes, torch
from weight_quantized_mixed_amd import qgemm as q
D = {D}
cache = q.KVCacheDesc(4096, 4096, 4, 16, 2, D)
x, t, pos, slots = torch.zeros((3, 64)).half(), torch.zeros((9, 0)), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
try:
    q.binding().append_norm(-1, 0, ctypes.addressof(cache), 2, D, x, x, x, t, t, pos, None, None, 1e-6, False, slots, None)
except ValueError as e:
    print("refused:", e)
"""


@pytest.mark.parametrize("D", [0, -1, -2**31])
def test_append_of_heads_without_places_is_refused(D):
    """A process of its own makes the call, since a division by such a size ends it."""
    pytest.importorskip("torch")
    q.binding()
    r = subprocess.run([sys.executable, "-c", CALL.format(D=D)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused: head_dim" in r.stdout, (r.returncode, r.stderr)
