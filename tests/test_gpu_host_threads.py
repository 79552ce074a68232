"""Two host threads whose calls raise a kernel's shared-memory limit at the same time: every later call still launches."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys, threading
import torch
from kv_cache_quantization_append_gb300 import QuantKVCache, lib

which = sys.argv[1]
B = 1000
cache = QuantKVCache(lib.make_config(1, 1, 1, B, 64, window=0), "cuda")
h = cache.handle
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
x = torch.zeros(B, 1, 1, 128, dtype=torch.bfloat16, device="cuda")
ln, par = i32(B), i32(B, 1) - 1
size = dict(tree=lib.kv_tree_scratch_bytes, decode=lambda h, l, b, n: lib.kv_decode_scratch_bytes(h, l, b))[which](h, 0, B, 1)
errors = []
both = threading.Barrier(2)


def work(me):
    s = torch.cuda.Stream()
    scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x) if which == "tree" else torch.empty(B, 1, 128, device="cuda")
    q = x if which == "tree" else x[:, :, 0]

    def call(b):
        try:
            if which == "tree":
                lib.kv_tree_attention(h, 0, x[:b], x[:b], q[:b], out[:b], ln[:b], par[:b], scratch, stream=s)
            else:
                lib.kv_decode_attention(h, 0, q[:b], out[:b], ln[:b], scratch, stream=s)
        except lib.KVQError as e:
            errors.append((b, str(e)))

    for b in range(2, B, 2):
        both.wait()
        call(b + me if b % 4 else b + 1 - me)    # one of them needs a little more than the other
        both.wait()
        call(b + 1)
    torch.cuda.synchronize()


threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, (len(errors), errors[:3])
"""


@pytest.mark.parametrize("which", ["tree", "decode"])
def test_two_threads_grow_the_shared_memory(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        done = subprocess.run([sys.executable, "-c", CODE, which], cwd=root, capture_output=True, text=True, timeout=300)
        assert done.returncode == 0, done.stderr[-1500:]
