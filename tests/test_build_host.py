"""What build() leaves behind where the serving extension cannot be built, and
when it is built again. Stand-ins for the sources: one small host file."""
import os

import pytest

from jagged_hstu_attention_gb300 import build_ext


@pytest.fixture
def small(tmp_path, monkeypatch):
    """build() of a one-file release library and extension under tmp_path."""
    lib, ext = str(tmp_path / "lib.so"), str(tmp_path / "_serving.so")
    monkeypatch.setattr(build_ext, "SOURCES", ["shard.cpp"])
    monkeypatch.setattr(build_ext, "VARIANTS", {"release": (lib, str(tmp_path / "obj"), [])})
    monkeypatch.setattr(build_ext, "EXT_PATH", ext)
    monkeypatch.setattr(build_ext, "EXT_STAMP", str(tmp_path / "obj" / "stamp"), raising=False)
    return lib, ext


def test_the_libraries_are_linked_where_the_extension_fails(small, monkeypatch):
    lib, ext = small

    def fails():
        raise RuntimeError("no Python.h")

    monkeypatch.setattr(build_ext, "_build_extension", fails)
    with open(ext, "w") as f:
        f.write("of an older torch")
    os.utime(ext, (0, 0))
    with pytest.warns(RuntimeWarning, match="no Python.h"):
        build_ext.build(variants=("release",))
    assert os.path.getsize(lib) > 0 and not os.path.exists(ext)
    before = os.path.getmtime(lib)
    with pytest.warns(RuntimeWarning, match="no Python.h"):  # tried again; the library is kept
        build_ext.build(variants=("release",))
    assert os.path.getmtime(lib) == before


def test_another_torch_builds_the_extension_again(small, monkeypatch):
    _, ext = small
    built = []

    def compiled(*args, **kwargs):
        built.append(args)
        with open(ext + ".tmp", "w") as f:
            f.write("extension")

        class Result:
            returncode, stdout, stderr = 0, "", ""
        return Result()

    run = build_ext.subprocess.run
    monkeypatch.setattr(build_ext.subprocess, "run",
                        lambda cmd, **kw: compiled(cmd) if cmd[0] == "g++" else run(cmd, **kw))
    version = "1.0"
    monkeypatch.setattr("importlib.metadata.version", lambda name: version)
    for want in (1, 1):
        build_ext.build(variants=("release",))
        assert len(built) == want
    version = "2.0"
    for want in (2, 2):
        build_ext.build(variants=("release",))
        assert len(built) == want
