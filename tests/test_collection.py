"""Every test that is written is collected: a module that defines a name twice
loses the first of the two, unless another name holds it."""

import ast
import glob
import os

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def lost(source):
    """Names of tests that a later definition replaces."""
    out, seen = [], {}  # name -> whether another test_ name holds it
    for node in ast.parse(source).body:
        if isinstance(node, (ast.FunctionDef, ast.ClassDef)):
            if node.name.lower().startswith("test") and seen.get(node.name) is False:
                out.append(node.name)
            seen[node.name] = False
        elif isinstance(node, ast.Assign) and isinstance(node.value, ast.Name) and node.value.id in seen:
            if any(isinstance(t, ast.Name) and t.id.startswith("test") for t in node.targets):
                seen[node.value.id] = True
    return out


@pytest.mark.parametrize("module", sorted(os.path.basename(f) for f in glob.glob(os.path.join(HERE, "*.py"))))
def test_no_test_replaces_another(module):
    with open(os.path.join(HERE, module)) as f:
        assert lost(f.read()) == []


def test_lost_names():
    two = "def test_a(): pass\n{}\ndef test_a(): pass\n"
    assert lost(two.format("")) == ["test_a"]
    assert lost(two.format("test_b = test_a")) == []
    assert lost(two.format("b = test_a")) == ["test_a"]
    assert lost("def f(): pass\ndef f(): pass\n") == []
