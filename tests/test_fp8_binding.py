"""The binding without its C part, and that part built without a DLPack header (CPU)."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "routed_expert_ffn_05_b200"
WITHOUT = f"import sys; sys.modules['{NAME}._marshal'] = None; "


def builder():
    spec = importlib.util.spec_from_file_location("moe_build", os.path.join(ROOT, NAME, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def run(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)


def test_the_package_works_without_its_c_part():
    r = run(WITHOUT + f"import {NAME} as M; assert M._marshal.__name__.endswith('marshal_py'); "
            "print(M.moe_workspace_size(M.make_dims(4, 256, 256, 8, 2)))")
    assert r.returncode == 0 and int(r.stdout) > 0, r.stderr


def test_the_host_tests_pass_without_the_c_part():
    r = run(WITHOUT + "import pytest; "
            "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', 'tests/test_fp8_host.py', 'tests/test_abi.py']))")
    assert r.returncode == 0, r.stdout[-3000:]


@pytest.mark.parametrize("include", [None, "torch"])
def test_the_c_part_builds_without_a_dlpack_header(tmp_path, include):
    """Built into a folder of its own and put in the package's place: the host tests, which look at tensors of every kind."""
    b = builder()
    target = str(tmp_path / "_marshal.so")
    assert b.build_marshal(target, b._torch_include() if include else None)
    bound = "True" if include else "False"
    r = run("import sys, importlib.util, torch; "
            f"s = importlib.util.spec_from_file_location('{NAME}._marshal', {target!r}); "
            f"m = importlib.util.module_from_spec(s); s.loader.exec_module(m); sys.modules['{NAME}._marshal'] = m; "
            f"assert m.bind(torch.Tensor, torch.nn.Parameter) is {bound}; import pytest; "
            "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', 'tests/test_fp8_host.py', "
            "'--deselect', 'tests/test_fp8_host.py::test_what_a_tensor_holds']))")
    assert r.returncode == 0, r.stdout[-3000:]


def test_a_build_without_torch_or_a_compiler_says_so_and_goes_on(tmp_path, monkeypatch, capsys):
    b = builder()
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert b._torch_include() is None
    target = str(tmp_path / "_marshal.so")
    open(target, "w").close()
    monkeypatch.setattr(b.subprocess, "run", lambda *a, **k: (_ for _ in ()).throw(FileNotFoundError("gcc")))
    assert b.build_marshal(target) is False and not os.path.exists(target)
    assert "gcc" in capsys.readouterr().err
