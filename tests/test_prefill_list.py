"""How the CTAs of a prefill over 8-bit blocks share its row tiles: every tile of every active one is taken once (CPU)."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from kv_cache_quantization_append_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
CTAS = 152


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("prefill_list") / "libprefill_list.so")
    subprocess.run([build.nvcc(), "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", os.path.join(HERE, "helpers", "prefill_list.cu"),
                    "-o", so], check=True)
    fn = ctypes.CDLL(so).walk
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 8 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]

    def call(pos, T, g, HL, W=64, bf16=True, max_seq_len=1 << 20, ctas=CTAS):
        pos = np.ascontiguousarray(pos, np.int32)
        room = len(pos) * HL * (T // (128 // g) + 1) + 2 * ctas
        out, info = np.zeros((room, 8), np.int32), np.zeros(2, np.int32)
        n = fn(pos.ctypes.data, len(pos), T, g, HL, W, 64 if bf16 else 32, max_seq_len, ctas, out.ctypes.data, room, info.ctypes.data)
        assert n >= 0
        return out[:n], bool(info[0]), int(info[1])

    return call


def _check(walk, pos, T, g, HL, W, bf16, **kw):
    out, whole, parts = walk(pos, T, g, HL, W, bf16, **kw)
    nx = -(-T // (128 // g))
    active = [b for b, p in enumerate(pos) if p >= 0 and p + T <= kw.get("max_seq_len", 1 << 20)]
    assert (parts > 0) == bool(active)
    at = {}
    for hl, b, x, ta, tb, n, cta, slot in out.tolist():
        assert 0 <= ta < tb <= n and cta < kw.get("ctas", CTAS)
        assert not whole or slot == -1
        at.setdefault((hl, b, x), []).append((ta, tb, n, cta, slot))
    assert sorted(at) == sorted((hl, b, x) for hl in range(HL) for b in active for x in range(nx))
    slots = set()
    for pieces in at.values():
        end = 0
        # in the order of the CTAs' records the pieces follow one another (the join adds them in that order)
        for ta, tb, n, cta, slot in sorted(pieces, key=lambda p: 2 * p[3] + max(p[4], 0)):
            assert ta == end
            end = tb
            if slot >= 0:
                assert (cta, slot) not in slots
                slots.add((cta, slot))
        assert end == pieces[0][2]
    return whole


@pytest.mark.parametrize("B", [9, 16, 32, 64])
@pytest.mark.parametrize("HL,g", [(1, 4), (2, 3), (8, 1), (8, 4)])
def test_one_active_sequence_anywhere(walk, B, HL, g):
    for T in (1, 16, 20, 33, 64, 100, 128):
        for p in (0, 50, 100, 1000):
            for s in range(B):
                pos = [-1] * B
                pos[s] = p
                _check(walk, pos, T, g, HL, 64, True)


def test_random_batches(walk):
    rng = np.random.default_rng(0)
    seen = [0, 0]
    for i in range(3000):
        B = int(np.exp(rng.uniform(0, np.log(100))))
        T = int(np.exp(rng.uniform(0, np.log(1500))))
        far = int(np.exp(rng.uniform(0, np.log(30000))))
        pos = np.where(rng.random(B) < rng.choice([0.1, 0.5, 1.0]), rng.integers(0, far + 1, B), -1)
        g, HL = int(rng.integers(1, 5)), int(rng.choice([1, 2, 4, 8, 24]))
        kw = dict(ctas=int(rng.choice([152, 148, 7, 1]))) if i % 4 == 0 else {}
        if i % 7 == 0:
            kw["max_seq_len"] = far // 2 + T
        seen[_check(walk, pos.tolist(), T, g, HL, int(rng.choice([32, 64, 100, 128, 1024])), bool(i % 2), **kw)] += 1
    assert min(seen) > 300


def test_nothing_to_do(walk):
    out, _, parts = walk([-1, -1], 5, 2, 4)
    assert len(out) == 0 and parts == 0
    out, _, parts = walk([100], 5, 2, 4, max_seq_len=104)
    assert len(out) == 0 and parts == 0


def test_one_long_sequence_among_many(walk):
    """Row tiles that are many are taken whole, but for one so long that its CTA would end after all others."""
    for far, whole in ((0, True), (20000, True), (100000, False)):
        for s in (0, 37, 63):
            pos = [0] * 64
            pos[s] = far
            assert _check(walk, pos, 256, 4, 8, 128, True) == whole
