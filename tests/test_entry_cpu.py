"""The script form of __graft_entry__.py: what it calls is defined before it runs."""
import ast
import os

from conftest import ROOT


def test_main_block_comes_last():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    mains = [i for i, s in enumerate(body) if isinstance(s, ast.If) and "__main__" in ast.dump(s.test)]
    assert mains == [len(body) - 1]


def test_smoke_reaches_its_last_part_as_a_script(monkeypatch):
    """The file run as a script, with stand-ins for the parts of smoke() that need a GPU: the calls of its last lines
    find their functions."""
    tree_file = os.path.join(ROOT, "__graft_entry__.py")
    with open(tree_file) as f:
        tree = ast.parse(f.read())
    called = []
    for s in tree.body:
        if not isinstance(s, ast.FunctionDef):
            continue
        if s.name == "smoke":  # only its calls of the file's own functions
            s.body = [x for x in s.body if isinstance(x, ast.Expr) and isinstance(x.value, ast.Call)
                      and getattr(x.value.func, "id", "").startswith("_smoke")]
            for x in s.body:
                x.value.args = []
            assert len(s.body) >= 2
        else:
            s.args.args, s.body = [], [ast.parse(f"called.append({s.name!r})").body[0]]
    monkeypatch.setattr("sys.argv", ["__graft_entry__.py", "smoke"])
    exec(compile(ast.fix_missing_locations(tree), "__graft_entry__.py", "exec"), 
         {"__name__": "__main__", "__file__": tree_file, "called": called})
    assert called == ["build", "_smoke_feed_forward", "_smoke_four_bits"]
