"""A copied tree runs its own kernels: the layer's binding finds the library beside it."""
import os
import shutil
import subprocess
import sys

import torch

import nvfp4_bit_block_gb300 as nv
from nvfp4_bit_block_gb300.build import BUILD, HERE, LAYER_EXT, LAYER_LIB

SHOW = """
import nvfp4_bit_block_gb300.layer as layer
layer._binding()
for line in sorted({l.split(None, 5)[-1].strip() for l in open("/proc/self/maps") if "nvfp4" in l}):
    print(line)
"""


def test_the_binding_of_a_copied_tree_loads_the_library_beside_it(tmp_path):
    nv.build()
    there = tmp_path / os.path.basename(HERE)
    (there / "_build").mkdir(parents=True)
    for name in os.listdir(HERE):
        if name.endswith(".py"):
            shutil.copy2(os.path.join(HERE, name), there)
    for lib in (LAYER_LIB, LAYER_EXT):
        shutil.copy2(lib, there / "_build")
    r = subprocess.run([sys.executable, "-c", SHOW], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    mapped = r.stdout.split("\n")[:-1]
    assert len(mapped) == 2 and all(m.startswith(str(there / "_build")) for m in mapped), mapped


def test_the_binding_is_linked_anew_for_another_torch(monkeypatch):
    """What it was built against is kept beside it."""
    nv.build()
    build_py = sys.modules["nvfp4_bit_block_gb300.build"]  # the package's own `build` is the function
    assert not build_py._ext_stale()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "x")
    assert build_py._ext_stale()
