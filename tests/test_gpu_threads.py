"""Calls from two threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Each size of shared memory is new to the process when two threads ask for it
# and for the next one.
GROWING = """
import threading, torch
from bit_packed_index_b200 import vq
ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
meet, errors = threading.Barrier(2), []
def work(odd):
    torch.cuda.set_device(0)
    for e in range(360, 1024, 2):
        meet.wait()
        try:
            vq.group_rows(ids, e + odd)
        except vq.VQError as err:
            errors.append((e + odd, str(err)))
threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
print(len(errors), errors[:3])
assert not errors
"""


def test_sizes_that_grow_in_two_threads():
    r = subprocess.run([sys.executable, "-c", GROWING], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]
