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


@pytest.mark.parametrize("error", [ImportError("No module named 'torch'"), FileNotFoundError(2, "g++"), RuntimeError("torch/csrc/Exceptions.h: not found")])
def test_library_is_built_where_the_module_cannot_be(error, monkeypatch, tmp_path, capsys):
    """Without PyTorch, a host compiler or headers the C library is linked all the same, and no older module stays beside it."""
    from weight_quantized_mixed_amd import build as b
    old = tmp_path / "_binding.so"
    old.write_bytes(b"older")
    commands = []

    def run(cmd):
        commands.append(cmd)
        if "-shared" in cmd:
            with open(cmd[cmd.index("-o") + 1], "wb"):
                pass
        return ""

    def fail():
        raise error

    for name, value in (("_run", run), ("build_binding", fail), ("BUILD", str(tmp_path / "objects")), ("LIB", str(tmp_path / "lib.so")),
                        ("BINDING", str(old))):
        monkeypatch.setattr(b, name, value)
    assert b.build() == str(tmp_path / "lib.so") and (tmp_path / "lib.so").exists()
    assert len(commands) == len(b.SOURCES) + 1
    assert not old.exists() and str(error) in capsys.readouterr().err


def test_missing_module_names_the_build(monkeypatch):
    monkeypatch.setattr(q, "_binding", None)
    monkeypatch.setitem(sys.modules, "weight_quantized_mixed_amd._binding", None)
    monkeypatch.delattr(sys.modules["weight_quantized_mixed_amd"], "_binding", raising=False)
    with pytest.raises(FileNotFoundError, match="weight_quantized_mixed_amd.build"):
        q.binding()
