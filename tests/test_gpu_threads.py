"""A fresh process whose first launches come from eight host threads at once, each on a stream
and workspace of its own and beginning with another call: every call gives what one thread
alone gets.  (A new thread has no CUDA context until a call of the runtime binds one.)"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import threading
import torch
import paged_kv_attention_17_gb300 as pkv
BF, N = torch.bfloat16, 8
g = torch.Generator("cuda").manual_seed(3)
normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
q, cache, table = normal(3, 16, 576), normal(40, 16, 576), torch.randperm(40, generator=g, device="cuda").int().view(2, 20)
wide, kv, rope = normal(200, 4, 192), normal(300, 4, 256), normal(300, 64)
qkv, pos = normal(70, 12, 128), torch.arange(70, device="cuda")
freq = (10000.0 ** (-torch.arange(64, device="cuda") / 64)).float()
kc, vc = normal(40, 16, 2, 128), normal(40, 16, 2, 128)
qsl, lens = ints(0, 1, 3), ints(300, 257)

def outputs():
    return [torch.zeros(3, 16, 512, dtype=BF, device="cuda"), torch.zeros(200, 4, 128, dtype=BF, device="cuda"),
            torch.zeros(70, 8, 128, dtype=BF, device="cuda"), torch.zeros(5, 16, 2, 128, dtype=BF, device="cuda"),
            torch.zeros(5, 16, 2, 128, dtype=BF, device="cuda"), torch.zeros(70, 8, 128, dtype=BF, device="cuda")]

def step(o, ws, mha_ws, first=0):
    calls = [
        lambda: pkv.pkv_latent_attention_varlen(q, cache, o[0], qsl, lens, table, 2, 320, 0.07, workspace=ws),
        lambda: pkv.pkv_expanded_attention_varlen(wide, kv[..., :128], rope, kv[..., 128:], o[1], ints_q, ints_k,
                                                  200, 300, 0.07),
        lambda: pkv.pkv_rotate_write(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], pos, freq, pos, o[2], o[3], o[4]),
        lambda: pkv.pkv_attention_varlen(qm, kc, vc, o[5], ints_m, lens, table, 40, 320, 0.09, workspace=mha_ws)]
    for k in range(4):
        calls[(first + k) % 4]()

qm = qkv[:, :8].contiguous()
ints_q, ints_k, ints_m = ints(0, 200), ints(0, 300), ints(0, 40, 70)
outs = [outputs() for _ in range(N + 1)]
ws = [torch.empty(64 << 20, dtype=torch.uint8, device="cuda") for _ in range(2 * N + 2)]
torch.cuda.synchronize()
gate, wrong = threading.Barrier(N), []

def work(i):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            gate.wait()
            for _ in range(5):
                step(outs[i], ws[2 * i], ws[2 * i + 1], i)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        wrong.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(N)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not wrong, wrong
step(outs[N], ws[2 * N], ws[2 * N + 1])
torch.cuda.synchronize()
for i in range(N):
    for a, b in zip(outs[i], outs[N]):
        assert torch.equal(a, b) and bool(a.any()), i
print("ok")
'''


def test_first_launches_of_eight_threads():
    got = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip().endswith("ok"), got.stderr[-2000:]
