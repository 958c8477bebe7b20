"""The indexer's entries need the C library alone: without the compiled part of the
serving operators' binding the package imports and they work, and a serving call
fails by name."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.modules["sparse_attention_indexer_quant_gb300._serving"] = None  # importing it fails
import torch
from sparse_attention_indexer_quant_gb300 import binding as idx
assert idx.lib.idx_version() >= 100
assert idx.paged_logits_topk_workspace_bytes(4, 1, 64, 2048) >= 0
assert idx.lib.idx_quant_insert(None, -1, 128, None, None, 1, 64, None, None) == 1
t = torch.zeros(1, dtype=torch.int32)
for call in (lambda: idx.plan_step(t, t, t[None], t, t, 1, 4), lambda: idx.rope_table(4, 8),
             lambda: idx.qk_norm_rope_insert(*[t] * 13), lambda: idx.paged_attention(t, t, t, t, t)):
    try:
        call()
    except RuntimeError as e:
        assert "serving binding" in str(e) and isinstance(e.__cause__, ImportError), e
    else:
        raise AssertionError("a serving call without its binding")
print("ok")
"""


def test_import_without_the_serving_binding():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


def test_the_library_is_linked_whatever_becomes_of_the_binding(tmp_path, monkeypatch):
    from sparse_attention_indexer_quant_gb300 import build_lib
    did = []

    def run(cmd, what):
        did.append(what)
        if what.startswith("g++"):
            raise RuntimeError("no headers")
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build_lib, "_run", run)
    monkeypatch.setattr(build_lib, "_sources", lambda: [])
    for name in ("BUILD", "LIB", "EXT"):
        monkeypatch.setattr(build_lib, name, str(tmp_path / name))
    with pytest.raises(RuntimeError, match="no headers"):
        build_lib.build(force=True)
    assert "link" in did and os.path.exists(tmp_path / "LIB") and not os.path.exists(tmp_path / "EXT")
