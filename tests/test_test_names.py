"""Two tests of one name in a module: the first would never be collected."""
import ast
import glob
import os

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def _lost(tree):
    """Top-level tests whose name is given to another test before anything else refers to it."""
    held, lost = set(), []
    for node in tree.body:
        if isinstance(node, ast.FunctionDef) and node.name.startswith("test"):
            if node.name in held:
                lost.append(node.name)
            held.add(node.name)
        elif isinstance(node, ast.Assign) and isinstance(node.value, ast.Name):
            held.discard(node.value.id)   # kept under another name
    return lost


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(HERE, "test_*.py"))), ids=os.path.basename)
def test_no_test_hides_another(path):
    with open(path) as f:
        assert _lost(ast.parse(f.read())) == []


def test_the_check_itself():
    twice = "def test_a():\n    pass\n\n\ndef test_a():\n    pass\n"
    assert _lost(ast.parse(twice)) == ["test_a"]
    assert _lost(ast.parse(twice.replace("\n\n\n", "\n\n\ntest_b = test_a\n\n\n"))) == []
