"""The build entry point works on a tree that has no built library yet."""
import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_build_file_runs_without_the_library(tmp_path):
    # a copy of the package without libwush.so: importing it fails, loading its build file does not
    pkg = tmp_path / "activation_quantization_b200"
    pkg.mkdir()
    for f in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(ROOT, "activation_quantization_b200", f), pkg / f)
    r = subprocess.run([sys.executable, "-c", "import activation_quantization_b200"], cwd=tmp_path,
                       capture_output=True, text=True)
    assert r.returncode != 0 and "build.py" in r.stderr
    code = "import runpy; assert callable(runpy.run_path('activation_quantization_b200/build.py')['build'])"
    subprocess.run([sys.executable, "-c", code], cwd=tmp_path, check=True)


def test_graft_build_does_not_import_the_package_first(tmp_path):
    # build() of a copy of the tree whose build.py only writes a marker, and whose package needs that marker
    pkg = tmp_path / "activation_quantization_b200"
    pkg.mkdir()
    shutil.copy(os.path.join(ROOT, "__graft_entry__.py"), tmp_path)
    (pkg / "build.py").write_text("import os\ndef build():\n    open(os.path.join(os.path.dirname(__file__), 'lib'), 'w')\n")
    (pkg / "__init__.py").write_text("import os\nassert os.path.exists(os.path.join(os.path.dirname(__file__), 'lib'))\n")
    subprocess.run([sys.executable, "-c", "import __graft_entry__ as g; g.build()"], cwd=tmp_path, check=True)
