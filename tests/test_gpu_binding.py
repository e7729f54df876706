"""The C++ binding on a GPU machine: its calls leave Python's lock to other threads."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = """
#include <unistd.h>
int vh_mrope_kv_append(void) { usleep(400000); return 0; }
int vh_window_decode_attn(void) { usleep(400000); return 0; }
int vh_window_prompt_attn(void) { usleep(400000); return 0; }
"""

SCRIPT = """
import sys, threading, time
sys.path.insert(0, %r)
import torch
import paged_len_decode_gb300 as v
z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
kc, table, row = z(4, 16, 2, 64, **bf), z(3, 2, **i32), z(3, **i32)
starts, ws = z(4, **i32), z(1 << 20, dtype=torch.uint8)
calls = dict(
    append=lambda: v.vh_mrope_kv_append(z(3, 4, 64, **bf), z(3, 2, 64, **bf), z(3, 2, 64, **bf), z(8, 64), kc, kc, table, row, row, z(3, 4, 64)),
    decode=lambda: v.vh_window_decode_attn(z(3, 4, 64), kc, kc, table, row, row, z(3, 4, 64, **bf), ws),
    prompt=lambda: v.vh_window_prompt_attn(z(5, 4, 64, **bf), kc, kc, table, starts, row, row, z(5, 4, 64, **bf), ws))
for name, call in calls.items():
    ticks, on = [0], True
    def count():
        while on:
            time.sleep(0.005)
            ticks[0] += 1
    t = threading.Thread(target=count)
    t.start()
    t0, before = time.time(), ticks[0]
    call()
    took, during = time.time() - t0, ticks[0] - before
    on = False
    t.join()
    print(name, took > 0.35, during > 10)
"""


def test_a_waiting_call_leaves_other_threads_running(tmp_path):
    """The C functions are replaced by ones that sleep, as a launch does where the queue is full."""
    src, lib = tmp_path / "stub.c", tmp_path / "stub.so"
    src.write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    r = subprocess.run([sys.executable, "-c", SCRIPT % ROOT], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, LD_PRELOAD=str(lib)))
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:3] == [f"{n} True True" for n in ("append", "decode", "prompt")], r.stdout
