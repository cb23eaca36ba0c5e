"""The entry script as a command: everything it calls is defined before its main block runs."""
import ast
from pathlib import Path

ENTRY = Path(__file__).resolve().parents[1] / "__graft_entry__.py"


def test_the_main_block_is_the_last_statement():
    body = ast.parse(ENTRY.read_text()).body
    mains = [i for i, x in enumerate(body) if isinstance(x, ast.If) and "__name__" in ast.unparse(x.test)]
    assert mains == [len(body) - 1]


def test_functions_that_the_script_calls_exist():
    tree = ast.parse(ENTRY.read_text())
    defined = {x.name for x in tree.body if isinstance(x, ast.FunctionDef)}
    called = {x.func.id for x in ast.walk(tree) if isinstance(x, ast.Call) and isinstance(x.func, ast.Name)}
    assert {"build", "smoke"} <= defined
    assert {x for x in called if x.startswith("_smoke")} <= defined
