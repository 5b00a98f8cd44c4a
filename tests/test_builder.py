"""The build of the torch front end beside the library: what stops the one does not stop the
other, and either is made again when, and only when, what it is made from has changed."""

import os

import pytest

from block_quantized_decode_rmsnorm_gb300 import builder

torch_dir = builder._torch_dir()
with_torch = pytest.mark.skipif(torch_dir is None, reason="torch with CUDA is not installed")


@pytest.fixture
def apart(tmp_path, monkeypatch):
    """The library as it is built, and a place for front ends of this test's own."""
    builder.build()
    monkeypatch.setattr(builder, "FRONT", str(tmp_path / os.path.basename(builder.FRONT)))
    monkeypatch.setattr(builder, "BUILD", str(tmp_path / "_build"))
    os.mkdir(builder.BUILD)
    monkeypatch.setattr(builder, "_build_library", lambda force, verbose: None)
    return monkeypatch


@with_torch
def test_a_front_end_that_fails_leaves_the_library(monkeypatch, tmp_path):
    builder.build()
    before = os.stat(builder.LIB).st_mtime_ns
    monkeypatch.setattr(builder, "FRONT", str(tmp_path / os.path.basename(builder.FRONT)))
    monkeypatch.setenv("CXX", "/bin/false")
    for _ in range(2):  # the second time as well: the library is not made again
        with pytest.warns(RuntimeWarning, match="front end"):
            assert builder.build() == builder.LIB
    with pytest.raises(RuntimeError, match="/bin/false"):
        builder.build(strict=True)
    monkeypatch.setenv("CXX", str(tmp_path / "no such compiler"))
    with pytest.warns(RuntimeWarning, match="no such compiler"):
        builder.build()
    assert os.stat(builder.LIB).st_mtime_ns == before and not os.path.exists(builder.FRONT)


def test_no_front_end_for_a_torch_without_cuda(apart, tmp_path):
    class Spec:
        origin = str(tmp_path / "torch" / "__init__.py")

    os.makedirs(tmp_path / "torch" / "lib")
    apart.setattr(builder.importlib.util, "find_spec", lambda name: Spec)
    apart.setenv("CXX", "/bin/false")
    builder.build(strict=True)
    apart.setattr(builder.importlib.util, "find_spec", lambda name: None)
    builder.build(strict=True)
    assert not os.path.exists(builder.FRONT)


@with_torch
def test_front_end_is_made_again_for_what_it_depends_on(apart):
    made = []

    def compile_front(*a):
        made.append(os.path.exists(builder.FRONT))
        open(builder.FRONT, "w").close()

    apart.setattr(builder, "_compile_front", compile_front)
    builder.build()
    builder.build()
    assert made == [False]
    apart.setenv("CXX", "another-c++")
    builder.build()
    apart.setattr(builder.sys, "implementation", type("", (), {"cache_tag": "cpython-399"}))
    builder.build()
    apart.setattr(builder.importlib.metadata, "version", lambda name: "99.0")
    builder.build()
    builder.build()
    assert made == [False] * 4  # each time without the older one
    builder.build(force=True)
    assert len(made) == 5
    os.remove(builder.FRONT)
    builder.build()
    assert len(made) == 6


@with_torch
def test_a_failed_front_end_is_not_an_older_one(apart):
    """Where it cannot be made again the older one goes, so that nobody takes it for this one."""
    def compile_front(*a):
        raise RuntimeError("no compiler")

    open(builder.FRONT, "w").close()
    apart.setattr(builder, "_compile_front", compile_front)
    with pytest.warns(RuntimeWarning):
        builder.build()
    assert not os.path.exists(builder.FRONT)


@with_torch
def test_a_torch_of_no_known_version_leaves_the_library(apart):
    def version(name):
        raise builder.importlib.metadata.PackageNotFoundError(name)

    apart.setattr(builder.importlib.metadata, "version", version)
    with pytest.warns(RuntimeWarning, match="front end"):
        assert builder.build() == builder.LIB
    with pytest.raises(ImportError):
        builder.build(strict=True)


def test_front_end_is_named_for_the_interpreter():
    import sysconfig

    assert builder.FRONT.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
