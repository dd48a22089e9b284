"""The host code of include/gdn_train.h (argument checks, workspace layout and
sizes, in gdnt_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer,
on the CPU: both API sources are recompiled with the sanitizers on the host
side only and linked with the device objects of the normal build, and the
host-side tests of that header run against the result.  The runs of the other
host code, and the canary, are test_sanitizers.py's."""
import glob
import os
import sys

import pytest

from test_sanitizers import CANARY, HIPCC, ROOT, SAN, _check_canary, _clean, _env, _run

API = ("gdn_api", "gdnt_api")


def test_training_host_api_under_address_and_undefined_sanitizers(tmp_path):
    rts = sorted(glob.glob("/opt/rocm/lib/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    objs = sorted(glob.glob(os.path.join(ROOT, "linear_attention_ssm_gdn_amd", "_build", "*.o")))
    dev_objs = [o for o in objs if os.path.basename(o) not in {a + ".o" for a in API}]
    if not rts or not os.path.exists(HIPCC):
        pytest.skip("hipcc or clang's AddressSanitizer runtime is not installed")
    if len(dev_objs) + len(API) != len(objs) or not dev_objs:
        pytest.skip("the library's objects are not built (run __graft_entry__.build())")
    host_san = [f for flag in SAN for f in ("-Xarch_host", flag)]
    src = tmp_path / "canary.cpp"
    src.write_text(CANARY.replace("malloc(8)", "(char*)malloc(8)"))
    _check_canary([HIPCC, "-O1", "-g", *host_san, str(src), "-o", str(tmp_path / "canary")], str(tmp_path / "canary"))

    san_objs = []
    for name in API:
        obj = tmp_path / (name + "_san.o")
        r = _run([HIPCC, "--offload-arch=gfx950", "-mcode-object-version=5", "-O1", "-g", "-std=c++17", "-fPIC",
                  "-fvisibility=hidden", *host_san, "-I" + os.path.join(ROOT, "include"), "-c",
                  os.path.join(ROOT, "linear_attention_ssm_gdn_amd", "csrc", name + ".cpp"), "-o", str(obj)])
        assert r.returncode == 0, r.stderr
        san_objs.append(str(obj))
    lib = tmp_path / "libgdn_san.so"
    r = _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *host_san, "-o", str(lib), *san_objs, *dev_objs])
    assert r.returncode == 0, r.stderr
    driver = (
        "import sys; sys.path[:0] = [%r, %r]\n"
        "import linear_attention_ssm_gdn_amd._lib as L; L.LIB_PATH = %r\n"
        "import pytest\n"
        "rc = pytest.main(['-q', '-x', '-p', 'no:cacheprovider', '-m', 'not gpu', 'tests/test_train_abi.py',\n"
        "                  'tests/test_train_workspace.py'])\n"
        "assert L.load()._name == %r, L.load()._name\n"
        "sys.exit(int(rc))\n" % (ROOT, os.path.join(ROOT, "tests"), str(lib), str(lib)))
    _clean(_run([sys.executable, "-c", driver], env=_env(rts[-1])))
