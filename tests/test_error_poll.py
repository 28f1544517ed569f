"""Error words are read and cleared in order with the calls around: the host sides of the library over a runtime without a
GPU (tests/fake_runtime.cpp)."""
import ctypes
import os
import subprocess
from pathlib import Path

import pytest

HERE = Path(__file__).resolve().parent


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from kv_cache_attention_ff_gb300 import build, ff
    at = tmp_path_factory.mktemp("fake")
    run = lambda *cmd: subprocess.run([str(x) for x in cmd], check=True, capture_output=True, text=True).stdout
    include = ["-I", build.INCLUDE, "-I", build.CSRC]
    flags = ["-O1", "-std=c++17", "-Xcompiler", "-fPIC", *include]
    for name in ("ff_paged", "ff_kv8", "ff_bank"):
        run(build._nvcc(), *build.ARCH, "-x", "cu", *flags, "-c", os.path.join(build.CSRC, f"{name}.cpp"), "-o", at / f"{name}.o")
    run(build._nvcc(), *flags, "-c", HERE / "fake_runtime.cpp", "-o", at / "fake.o")
    # what is not called here, or has nothing to answer but that it went well
    objects = sorted(at.glob("*.o"))
    names = lambda what: {x.split()[-1] for x in run("nm", what, *objects).splitlines() if x and not x.endswith(":")}
    missing = names("--undefined-only") - names("--defined-only")
    missing = sorted(x for x in missing if x.startswith(("cuda", "__cuda", "_ZN2ff")))
    (at / "rest.c").write_text("".join(f"long {x}(void) {{ return 0; }}\n" for x in missing))
    run("gcc", "-w", "-fPIC", "-fno-builtin", "-c", at / "rest.c", "-o", at / "rest.o")
    # another runtime may be loaded for all (torch's): its functions are not meant
    run("g++", "-shared", "-Wl,-Bsymbolic", "-o", at / "fake.so", *objects, at / "rest.o")
    lib = ctypes.CDLL(str(at / "fake.so"))
    lib.fake_log.restype = ctypes.c_char_p
    lib.ff = ff
    return lib


@pytest.fixture(params=["ff_paged", "ff_kv8", "ff_bank"])
def handle(lib, request):
    kind = request.param
    desc = {"ff_paged": lib.ff.PagedDesc, "ff_kv8": lib.ff.KV8Desc, "ff_bank": lib.ff.BankDesc}[kind]()
    default = "ff_desc_default" if kind == "ff_bank" else f"{kind}_desc_default"
    assert getattr(lib, default)(ctypes.byref(desc)) == 0
    if kind == "ff_bank":
        desc.n_layers = desc.n_stages = 1
        desc.frame_h = desc.frame_w = 4
    else:
        desc.capacity = 100
    h = ctypes.c_void_p()
    assert getattr(lib, f"{kind}_create")(ctypes.byref(desc), ctypes.byref(h)) == 0
    yield kind, h
    assert getattr(lib, f"{kind}_destroy")(h) == 0


def poll(lib, handle, word):
    lib.fake_clear()
    lib.fake_word(word)
    rc = getattr(lib, f"{handle[0]}_error_poll")(handle[1])
    return rc, lib.fake_log().decode().split()


def test_nothing_to_report(lib, handle):
    rc, calls = poll(lib, handle, 0)
    assert rc == 0 and calls == ["wait"]


@pytest.mark.parametrize("word", [1, 2, 3])
def test_the_word_is_cleared_before_the_call_returns(lib, handle, word):
    """A later call's kernels, on streams that do not wait for the legacy one, neither meet what is being cleared nor
    lose what they report to it."""
    if handle[0] == "ff_bank" and word != 1:
        pytest.skip("a bank drops no rows")
    rc, calls = poll(lib, handle, word)
    assert rc == (6 if word & 1 else 8)
    assert calls[0] == calls[-1] == "wait" and "memset" in calls
    if handle[0] == "ff_paged" and word & 1:  # the counts of finished key ranges, too
        assert calls.count("memset") == 2
    assert poll(lib, handle, 0) == (0, ["wait"])
