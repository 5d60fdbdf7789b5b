"""The README's Python block reads as one program: its calls exist, and no name stands for two things."""
import ast
import os
import re

import adapter_sgmv_bgmv_gb300 as L

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_python_block():
    with open(PATH) as f:
        tree = ast.parse(re.search(r"```python\n(.*?)```", f.read(), re.S).group(1))
    made = {}
    for node in tree.body:
        if isinstance(node, ast.Assign) and isinstance(node.value, ast.Call) and isinstance(node.targets[0], ast.Name):
            made.setdefault(node.targets[0].id, set()).add(ast.unparse(node.value.func))
    assert made["ctx"] == {"L.Context"}
    assert {k: v for k, v in made.items() if len(v) > 1} == {}
    for node in ast.walk(tree):
        if isinstance(node, ast.Attribute) and isinstance(node.value, ast.Name):
            name = node.value.id
            if name == "L":
                assert hasattr(L, node.attr), node.attr
            elif name in made:
                func = next(iter(made[name]))              # L.Class or L.Class.maker
                assert hasattr(getattr(L, func.split(".")[1]), node.attr), f"{name}.{node.attr}"
