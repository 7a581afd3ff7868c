"""No test is lost to another of the same name in its file: the later definition
rebinds the name, and pytest collects the later one alone."""
import ast
import glob
import os

import pytest

from conftest import ROOT

FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(ROOT, "tests", "test_*.py")))


def lost(tree):
    """Names of module-level tests that are defined again without a second
    name given to the first definition before."""
    bound, kept, out = set(), set(), []
    for node in tree.body:
        if isinstance(node, ast.FunctionDef) and node.name.startswith("test"):
            if node.name in bound and node.name not in kept:
                out.append(node.name)
            bound.add(node.name)
            kept.discard(node.name)
        elif isinstance(node, ast.Assign) and isinstance(node.value, ast.Name):
            if any(isinstance(t, ast.Name) and t.id.startswith("test") for t in node.targets):
                kept.add(node.value.id)
    return out


@pytest.mark.parametrize("name", FILES)
def test_every_test_is_collected(name):
    with open(os.path.join(ROOT, "tests", name)) as f:
        assert lost(ast.parse(f.read())) == []
