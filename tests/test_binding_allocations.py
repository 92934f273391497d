"""Outputs that the binding allocates have the type that the library writes, whatever torch's default type is."""
import ast
import inspect

from sinkhorn_point_cloud_gb300 import binding


def test_every_allocation_names_its_type():
    calls = [n for n in ast.walk(ast.parse(inspect.getsource(binding))) if isinstance(n, ast.Call)]
    made = [n for n in calls if ast.unparse(n.func) in ("torch.empty", "torch.zeros", "torch.ones", "torch.full", "torch.tensor")]
    assert made
    for n in made:
        assert "dtype" in [k.arg for k in n.keywords], ast.unparse(n)
