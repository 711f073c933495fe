"""CPU test of the README's examples: a connection has to outlive the work queued
on it, so each one that an example opens is kept in a name, and closed only
behind a synchronisation."""
import ast
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "README.md")) as f:
    EXAMPLES = re.findall(r"```python\n(.*?)```", f.read(), re.S)


def called(node):
    return ast.unparse(node.func).split(".")[-1] if isinstance(node, ast.Call) else None


def test_there_are_examples():
    assert len(EXAMPLES) >= 2


@pytest.mark.parametrize("text", EXAMPLES, ids=range(len(EXAMPLES)))
def test_connections_are_kept(text):
    tree = ast.parse(text)
    opened = [n for n in ast.walk(tree) if called(n) in ("Conn", "make_conn")]
    kept = [s.value for s in tree.body if isinstance(s, ast.Assign)]
    assert opened and all(n in kept for n in opened)


@pytest.mark.parametrize("text", EXAMPLES, ids=range(len(EXAMPLES)))
def test_connections_are_closed_behind_a_synchronisation(text):
    order = [called(s.value) for s in ast.parse(text).body if isinstance(s, ast.Expr)]
    assert "close" in order and order[order.index("close") - 1] == "synchronize"
