"""The extension behind the serving-step calls is needed by those calls alone, and only
the one for this Python and this torch is loaded (no GPU)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

PACKAGE = "paged_kv_cache_96_gb300"


@pytest.fixture(scope="module")
def built():
    from paged_kv_cache_96_gb300 import build
    build.build()
    return build


def run(root, code):
    env = dict(os.environ, PYTHONPATH=str(root))
    env.pop("PA_LIBRARY", None)
    return subprocess.run([sys.executable, "-c", code], cwd=root, env=env, capture_output=True,
                          text=True)


OLDER_CALLS = """
import torch
{change}
from paged_kv_cache_96_gb300 import binding as B
assert B.pa_decode_workspace_bytes(1, 8, 2, 64, 1000, 256) > 0
bm = B.BlockManager(8, 16, 4)
bm.add_sequence(0)
bm.append_tokens(0, 20)
assert len(bm.table(0)) == 2
"""

NEW_CALLS = """
i, x = torch.zeros(1, dtype=torch.int32), torch.zeros(1)
for call in (lambda: B.pa_build_step_maps(*[i] * 5, 16, 8, *[i] * 6),
             lambda: B.pa_rope_and_cache(*[x] * 9),
             lambda: B.pa_decode_attention_window(*[x] * 6, 1, 0.1, 4),
             lambda: B.pa_prefill_attention_window(*[x] * 7, 1, 0.1, 4)):
    try:
        call()
    except {error}:
        pass
    else:
        raise SystemExit("no error")
"""


def test_other_calls_need_no_extension(built, tmp_path):
    """Without the extension the package imports and its ctypes calls answer; the
    serving-step calls say what is missing."""
    shutil.copytree(os.path.join(built.HERE), tmp_path / PACKAGE,
                    ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
    os.symlink(built.LIB, tmp_path / PACKAGE / "lib" / os.path.basename(built.LIB))
    code = OLDER_CALLS.format(change="") + NEW_CALLS.format(error="ImportError")
    r = run(tmp_path, code)
    assert r.returncode == 0, r.stdout + r.stderr


def test_extension_of_another_torch_is_not_loaded(built):
    """Under a torch that the extension was not built for, the others work on."""
    code = OLDER_CALLS.format(change="torch.__version__ = '1.2.3+other'") + \
        NEW_CALLS.format(error="ImportError") + \
        "assert not any('/_calls' in line for line in open('/proc/self/maps'))\n"
    r = run(os.path.dirname(built.HERE), code)
    assert r.returncode == 0, r.stdout + r.stderr


def test_extension_is_loaded_on_first_use(built):
    code = OLDER_CALLS.format(change="") + \
        "assert not any('/_calls' in line for line in open('/proc/self/maps'))\n" + \
        NEW_CALLS.format(error="ValueError") + \
        "assert any('/_calls' in line for line in open('/proc/self/maps'))\n"
    r = run(os.path.dirname(built.HERE), code)
    assert r.returncode == 0, r.stdout + r.stderr


def test_name_says_what_it_was_built_for(built):
    import torch
    path = built.calls_path(torch.__version__)
    assert os.path.exists(path)
    assert path.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__ in path
    assert built.calls_path("1.2.3") != path


def test_library_is_built_where_the_extension_does_not_compile(built, monkeypatch, tmp_path):
    def no_compiler():
        raise RuntimeError("no host compiler")
    monkeypatch.setattr(built, "HERE", str(tmp_path))
    monkeypatch.setattr(built, "_build_calls", no_compiler)
    monkeypatch.setattr(built, "library_up_to_date", lambda: True)
    with pytest.warns(UserWarning, match="no host compiler"):
        assert built.build() == built.LIB


def test_extension_of_older_sources_does_not_stay(built, monkeypatch, tmp_path):
    """Where it is out of date and does not compile there is none, rather than one that
    passes the library other arguments."""
    (tmp_path / os.path.basename(built.calls_path("1.2.3"))).touch()
    (tmp_path / "_calls.so").touch()

    def no_compiler():
        raise RuntimeError("no host compiler")
    monkeypatch.setattr(built, "HERE", str(tmp_path))
    monkeypatch.setattr(built, "_build_calls", no_compiler)
    monkeypatch.setattr(built, "library_up_to_date", lambda: True)
    with pytest.warns(UserWarning, match="no host compiler"):
        built.build()
    assert not os.listdir(tmp_path)
