"""What a build makes and when: the library does not wait for, nor change with, what only the binding needs.  Compilers are
stood in for by functions that write the file they are asked for."""
import os
import types

import pytest

from attention_flash_attn_gb300 import build as b


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    """A build of this tree's sources into an empty place; returns what was run, in order."""
    ran = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        what = "binding" if "g++" in cmd[0] else "lib"
        step = f"{what} {'link' if '-shared' in cmd else 'compile'}"
        ran.append(step)
        fails = step in run.fails
        if not fails:
            with open(out, "w") as f:
                f.write("x")
        return types.SimpleNamespace(returncode=int(fails), stdout="", stderr="no headers" if fails else "")

    run.fails = set()
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    for name, at in (("BUILD", "_build"), ("LIB", "lib.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    ran_and = types.SimpleNamespace(ran=ran, run=run)
    return ran_and


def test_everything_is_made_once(tree):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.BINDING)
    assert sorted(set(tree.ran)) == ["binding compile", "binding link", "lib compile", "lib link"]
    assert tree.ran.index("lib link") < tree.ran.index("binding link")
    tree.ran.clear()
    b.build()
    assert tree.ran == []


def test_the_library_is_made_where_the_binding_cannot_be(tree):
    tree.run.fails.add("binding compile")
    with pytest.raises(RuntimeError, match="no headers"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING) and "lib link" in tree.ran
    tree.run.fails.clear()
    tree.ran.clear()
    b.build()  # and then nothing of it again
    assert tree.ran == ["binding compile", "binding link"] and os.path.exists(b.BINDING)


def test_another_pytorch_recompiles_the_binding_alone(tree, monkeypatch):
    b.build()
    tree.ran.clear()
    monkeypatch.setattr(b.torch, "__version__", "0.0")
    b.build()
    assert tree.ran == ["binding compile", "binding link"]
