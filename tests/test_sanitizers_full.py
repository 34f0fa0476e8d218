"""Host sanitizer run (no GPU) of the full-attention layers' C ABI validation: built with
AddressSanitizer and UndefinedBehaviorSanitizer for the host, driven by
tests/sanitize/full_abi_driver.cpp. The kernels themselves are not instrumented;
the driver only makes calls that are rejected, are no-ops or are size queries."""
import os

import pytest

from test_sanitizers import ENV, HIPCC, ROOT, SAN, run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_full_abi_validation_under_address_and_ub_sanitizers(tmp_path):
    from gated_delta_rule_22_amd import _build
    objs = [os.path.join(_build.BUILD, s.rsplit(".", 1)[0] + ".o") for s in _build.SOURCES
            if s != "kda_full_api.cpp"]
    if not all(os.path.exists(o) for o in objs):
        _build.build()
    # host-side instrumentation only: each sanitizer flag goes to the host pass
    host_san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"):
        host_san += ["-Xarch_host", flag]
    common = [f"--offload-arch={_build.ARCH}", "-O1", "-g", "-std=c++17", "-fPIC",
              "-I", os.path.join(ROOT, "include"), "-I", _build.CSRC, "-I", _build.CSRC_SERVE, *host_san]
    api, drv, exe = (tmp_path / n for n in ("full_api_san.o", "driver.o", "full_abi_driver"))
    run([HIPCC, *common, "-x", "hip", "-c", os.path.join(_build.CSRC_SERVE, "kda_full_api.cpp"),
         "-o", str(api)])
    run([HIPCC, *common, "-c", os.path.join(SAN, "full_abi_driver.cpp"), "-o", str(drv)])
    run([HIPCC, f"--offload-arch={_build.ARCH}", *host_san, str(drv), str(api), *objs, "-o", str(exe)])
    r = run([str(exe)], env=ENV, timeout=120)
    assert "\n0 failures" in r.stdout, r.stdout
