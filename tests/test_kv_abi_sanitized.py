"""The validation and sizing paths of include/snip_kv.h under AddressSanitizer
and UndefinedBehaviorSanitizer (host code): tests/helpers/abi_asan_kv_check,
built from the library's sources and tests/helpers/abi_asan_kv_check.cpp by
sub_byte_mixed_amd/build.py (build_asan_check); none of its calls reaches the
GPU."""
import json
import os
import re
import subprocess

HELPERS = os.path.join(os.path.dirname(os.path.abspath(__file__)), "helpers")
BIN = os.path.join(HELPERS, "abi_asan_kv_check")


def test_cache_calls_clean_under_asan_and_ubsan():
    if not os.path.exists(BIN):
        from sub_byte_mixed_amd import build
        build.build_asan_check()
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([BIN], capture_output=True, text=True, timeout=120, env=env)
    assert "ERROR: AddressSanitizer" not in res.stderr, res.stderr[-4000:]
    assert "runtime error" not in res.stderr, res.stderr[-4000:]
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]
    out = json.loads(res.stdout.strip().splitlines()[-1])
    assert out["failures"] == 0 and out["sized"] > 0


def test_the_sanitized_check_calls_every_entry_point():
    root = os.path.dirname(os.path.dirname(HELPERS))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "snip_kv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(snipkv_[a-z0-9_]+)\s*\(", text))
    used = set(re.findall(r"\b(snipkv_[a-z0-9_]+)\s*\(", open(os.path.join(HELPERS, "abi_asan_kv_check.cpp")).read()))
    assert names <= used, sorted(names - used)
