"""Building and loading: the C library needs no torch, the decode operators' extension belongs to one
version of it."""
import os
import shutil
import subprocess
import sys

import pytest

import block_scaled_fp8_weight_gb300 as bsf8
from block_scaled_fp8_weight_gb300 import build as bsf8_build

NAME = "block_scaled_fp8_weight_gb300"
NO_TORCH = "import sys; sys.modules['torch'] = None; "  # importing it raises ImportError


@pytest.fixture(scope="module")
def alone(tmp_path_factory):
    """A tree with the sources and a good libbsf8.so, and no extension."""
    bsf8_build.build()
    root = tmp_path_factory.mktemp("tree")
    shutil.copytree(bsf8_build.HERE, root / NAME, ignore=shutil.ignore_patterns("_bsf8_torch*", "_build", "__pycache__"))
    shutil.copytree(bsf8_build.INCLUDE, root / "include")
    lib = root / NAME / "libbsf8.so"
    os.utime(lib)
    return root


def run(root, code):
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)


def test_the_library_is_loaded_without_torch_or_the_extension(alone):
    r = run(alone, NO_TORCH + f"import {NAME} as b; print(b.load(build_if_missing=False).bsf8_version(), b.library_path())")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[1] == str(alone / NAME / "libbsf8.so")


def test_the_library_is_built_without_torch(alone):
    r = run(alone, NO_TORCH + f"from {NAME} import build as b; assert b.up_to_date(); print(b.build())")
    assert r.returncode == 0 and r.stdout.strip() == str(alone / NAME / "libbsf8.so"), r.stderr
    # stale: as far as the first compiler call
    code = NO_TORCH + (f"from {NAME} import build as b; import subprocess as s; told = []\n"
                       "def f(cmd, **kw): told.append(cmd[0]); raise KeyError('compiler called')\n"
                       "s.run = f\n"
                       "try: b.build(force=True)\n"
                       "except KeyError: print(len(told) > 0 and all('nvcc' in x for x in told))")
    r = run(alone, code)
    assert r.returncode == 0 and r.stdout.strip() == "True", r.stderr


def test_names_are_there_without_torch(alone):
    r = run(alone, NO_TORCH + f"from {NAME} import *; print(KVCache, MAX_NODES, qkv_append, kv_commit, gemm)")
    assert r.returncode == 0, r.stderr
    assert not any(f.startswith("_bsf8_torch") for f in os.listdir(alone / NAME))


def test_an_extension_for_another_torch_is_not_taken(monkeypatch):
    torch = pytest.importorskip("torch")
    mine = bsf8_build.build_extension()
    assert os.path.exists(mine) and bsf8_build.extension_path() == mine
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    assert bsf8_build.extension_path() != mine and not os.path.exists(bsf8_build.extension_path())
    monkeypatch.setattr(bsf8_build, "_extension", None)
    with pytest.raises(RuntimeError, match="not built for this torch"):
        bsf8_build.load_extension(build_if_missing=False)


def test_every_name_is_exported():
    for name in bsf8.__all__:
        assert getattr(bsf8, name) is not None
