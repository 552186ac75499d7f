"""First calls from several host threads at once, in a process of their own: what a call sets up once per process is set up
right, whichever thread comes first."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import threading
import torch
import paged_kv_cache_409_b200 as pkv
from int8_helpers import make_pools

lens, ns = [700, 90], [3, 40]
kp, vp, bt = make_pools(lens, 16, 2, 128, seed=1)
bt = torch.cat([bt, bt.new_full((2, 4000), -1)], 1).contiguous()
q = torch.randn(43, 4, 128, device='cuda').half()
cl = torch.tensor(lens, dtype=torch.int32, device='cuda')
qsl = torch.tensor([0, 3, 43], dtype=torch.int32, device='cuda')
ws = [torch.empty(1 << 26, dtype=torch.uint8, device='cuda') for _ in range(8)]
kf, vf = (torch.randn(kp.shape[0], 16, 2, 128, device='cuda').half() for _ in range(2))
torch.cuda.synchronize()

def decode(call, k, v, i):  # parts of 16 to 16 * 4000 tokens: another amount of shared memory each
    out = torch.empty_like(q[:2])
    call(out, q[:2], k, v, bt, cl, 0.1, 60000, partition_size=16 * (1, 4000, 30, 2500, 7, 3600, 90, 1800)[i], workspace=ws[i])
    return out

def prefill(i):
    out = torch.empty_like(q)
    pkv.paged_attention_prefill_chunk_int8(out, q, kp, vp, bt, cl, qsl, 40, 0.1)
    return out

for what in (lambda i: decode(pkv.paged_attention_decode_int8, kp, vp, i), lambda i: decode(pkv.paged_attention_decode, kf, vf, i),
             prefill):
    got, gate = [None] * 8, threading.Barrier(8)
    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            got[i] = what(i)
            torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for i in range(8):
        again = what(i)
        torch.cuda.synchronize()
        assert got[i] is not None and torch.equal(got[i], again), i
assert pkv.get_device_error() == 0
print('agreed')
"""


def test_first_calls_of_eight_threads():
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", CODE], env=env, capture_output=True, text=True, timeout=200)
        assert r.returncode == 0 and "agreed" in r.stdout, r.stdout + r.stderr
