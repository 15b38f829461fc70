"""The build and smoke entry points run as a script: everything they call is defined before they are called."""
import ast
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRY = os.path.join(ROOT, "__graft_entry__.py")


def test_script_reaches_every_function_it_calls(tmp_path):
    """Run as a script with its functions' bodies reduced to the calls of one another."""
    tree = ast.parse(open(ENTRY).read())
    names = {n.name for n in tree.body if isinstance(n, ast.FunctionDef)}
    assert {"build", "smoke"} <= names
    for f in tree.body:
        if isinstance(f, ast.FunctionDef):
            called = sorted({n.func.id for n in ast.walk(f) if isinstance(n, ast.Call) and isinstance(n.func, ast.Name)} & names)
            f.args = ast.parse("def f(*a): pass").body[0].args
            f.body = ast.parse("\n".join([f"print({f.name!r})"] + [f"{c}()" for c in called])).body
    script = tmp_path / "entry.py"
    script.write_text(ast.unparse(ast.fix_missing_locations(tree)))
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert set(r.stdout.split()) == names

