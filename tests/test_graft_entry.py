"""`python __graft_entry__.py smoke` runs what the imported module's smoke() runs."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_command_comes_after_all_that_it_calls():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    commands = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__name__" in ast.unparse(node.test)]
    assert commands == [len(body) - 1], [ast.unparse(n).splitlines()[0] for n in body[commands[0] + 1:]]
