"""__graft_entry__.py run as a script: everything that it may call is defined
before it is called."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_script_ends_with_its_main_guard():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    guards = [i for i, node in enumerate(body)
              if isinstance(node, ast.If) and "__name__" in ast.unparse(node.test)]
    assert guards == [len(body) - 1]
