"""The prompt planner's and the block tables' host code under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): the host test files of both run in a child
process against libgk_san.so."""
import sys

from test_sanitizers_host import _run

HOST_TESTS = ["tests/test_prompt_host.py", "tests/test_tables_host.py"]


def test_prompt_and_tables_host_code_under_sanitizers():
    from paged_kv_cache_pool_gb300 import build
    build.build()
    build.build_sanitized()
    rc, out = _run([sys.executable, "-m", "pytest", *HOST_TESTS, "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu"],
                   build.sanitizer_env())
    assert rc == 0, out
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out
