"""The README's snippets: each call of the package exists and takes the arguments given."""
import ast
import inspect
import os
import re

import pytest

import entropy_logits_bf16_gb300 as rlk

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def calls():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return [node for block in blocks for node in ast.walk(ast.parse(block)) if isinstance(node, ast.Call)
            and isinstance(node.func, ast.Attribute) and isinstance(node.func.value, ast.Name) and node.func.value.id == "rlk"]


CALLS = calls()


def test_there_are_some():
    assert len(CALLS) >= 8


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.func.attr)
def test_call_binds(call):
    """As the interpreter would bind it; required keywords and misplaced positions show."""
    args, kwargs = [ast.unparse(a) for a in call.args], {k.arg: ast.unparse(k.value) for k in call.keywords}
    bound = inspect.signature(getattr(rlk, call.func.attr)).bind(*args, **kwargs).arguments
    for name, text in bound.items():   # a variable named like a parameter stands in its place
        if text in inspect.signature(getattr(rlk, call.func.attr)).parameters:
            assert text == name
    for node in ast.walk(call):        # constants exist
        if isinstance(node, ast.Attribute) and isinstance(node.value, ast.Name) and node.value.id == "rlk":
            assert hasattr(rlk, node.attr)
