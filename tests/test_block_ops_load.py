"""The compiled module of the operators when it cannot be imported."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


# the import of the compiled module fails: it is not there, or it does not load
FAILS = """
import sys, importlib.abc
class Finder(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path, target=None):
        if name == "weight_only_bit_moe_amd._block_ops":
            raise {error}
sys.meta_path.insert(0, Finder())
import weight_only_bit_moe_amd as M
try:
    M.add_rmsnorm
except RuntimeError as e:
    print(e)
"""


def test_a_module_that_is_not_built_is_named():
    r = run(FAILS.format(error="ModuleNotFoundError('No module named ' + repr(name), name=name)"))
    assert "_block_ops is missing: build it" in r.stdout, r.stdout + r.stderr


def test_a_module_that_does_not_load_says_why():
    r = run(FAILS.format(error="ImportError('undefined symbol: some_symbol_of_another_torch')"))
    assert "undefined symbol: some_symbol_of_another_torch" in r.stdout, r.stdout + r.stderr
    assert "missing" not in r.stdout and "build" in r.stdout
