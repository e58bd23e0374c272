"""The scripts at the root run as programs: what they call is defined before the
`if __name__ == "__main__"` that ends the file."""
import ast
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["__graft_entry__.py", "bench.py"])
def test_nothing_follows_the_main_guard(name):
    with open(os.path.join(ROOT, name)) as f:
        body = ast.parse(f.read()).body
    guards = [i for i, x in enumerate(body)
              if isinstance(x, ast.If) and ast.unparse(x.test) == "__name__ == '__main__'"]
    assert guards == [len(body) - 1]
