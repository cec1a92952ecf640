"""build() of __graft_entry__.py: the library's build does not hang on files of its tests."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STEP = "def build(verbose=False):\n    print('built {}')\n"


@pytest.mark.parametrize("checks", [(), ("build",), ("build", "build_cache")], ids=["none", "one", "both"])
def test_build_with_the_checks_that_are_there(tmp_path, checks):
    """The entry file over steps that only say their name, with none, one and both of the C checks' build files."""
    (tmp_path / "__graft_entry__.py").write_text(open(os.path.join(ROOT, "__graft_entry__.py")).read())
    steps = [("oracle", "build"), ("copy_reduce_amd", "build")] + [(os.path.join("tests", "capi"), c) for c in checks]
    for folder, name in steps:
        (tmp_path / folder).mkdir(parents=True, exist_ok=True)
        (tmp_path / folder / (name + ".py")).write_text(STEP.format(folder + "/" + name))
    (tmp_path / "copy_reduce_amd" / "__init__.py").write_text("")
    r = subprocess.run([sys.executable, "-c", "import __graft_entry__ as g; g.build()"], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split("\n")[:-1] == [f"built {folder}/{name}" for folder, name in steps]
