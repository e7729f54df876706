"""The package without its C++ binding, and when the binding is built anew (no GPU)."""
import importlib.util
import os
import subprocess
import sys


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.path.insert(0, %r)
class Hide:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._vh_bind"):
            raise ImportError("undefined symbol: xyz")
sys.meta_path.insert(0, Hide())
import paged_len_decode_gb300 as v
print(v.vh_status_string(v.VH_EINVAL) != "", v.vh_decode_workspace_bytes(4, 16, 8, 128, 16, 4) > 0, v.vh_prompt_workspace_bytes(9, 2, 4, 2, 64))
for call in (v.vh_mrope_kv_append, v.vh_window_decode_attn, v.vh_window_prompt_attn):
    try:
        call(1, 2, out=3)
    except ImportError as e:
        print(call.__name__, call.__name__ in str(e), "undefined symbol: xyz" in str(e))
"""


def test_other_calls_work_without_the_binding():
    r = subprocess.run([sys.executable, "-c", SCRIPT % ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:4] == ["True True 256"] + [
        f"{n} True True" for n in ("vh_mrope_kv_append", "vh_window_decode_attn", "vh_window_prompt_attn")], r.stdout


def build_script():
    spec = importlib.util.spec_from_file_location("_vh_build_test", os.path.join(ROOT, "paged_len_decode_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_binding_is_stale_after_another_torch(tmp_path, monkeypatch):
    b = build_script()
    src, obj, stamp = (str(tmp_path / n) for n in ("bind.cpp", "bind.o", "bind.stamp"))
    for f in (src, obj):
        open(f, "w").close()
    assert b._bind_stale(obj, [src], stamp)                       # built before there was a stamp
    with open(stamp, "w") as f:
        f.write(b._bind_stamp())
    assert not b._bind_stale(obj, [src], stamp)
    os.utime(src, (os.path.getmtime(obj) + 5,) * 2)
    assert b._bind_stale(obj, [src], stamp)                       # the source is newer
    os.utime(src, (os.path.getmtime(obj) - 5,) * 2)
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text("__version__ = '9.9'\n")
    monkeypatch.setattr(b, "_torch_dir", lambda: str(other))
    assert b._bind_stale(obj, [src], stamp)                       # another torch
    with open(stamp, "w") as f:
        f.write(b._bind_stamp())
    assert not b._bind_stale(obj, [src], stamp)
    (other / "version.py").write_text("__version__ = '9.10'\n")
    assert b._bind_stale(obj, [src], stamp)                       # the same place, another version


def test_build_compiles_a_stale_binding_only(monkeypatch, tmp_path):
    b = build_script()
    b.build()
    compiled = []
    monkeypatch.setattr(b, "_compile_bind", lambda src, obj, stamp: compiled.append(obj) or "")
    b.build()
    assert compiled == []
    monkeypatch.setattr(b, "_bind_stamp", lambda: "another")
    b.build()
    assert len(compiled) == 1
