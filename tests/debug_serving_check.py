"""Run by tests/test_debug_serving_gpu.py in a child process whose FA_LIBRARY points
at the bounds-checked build: the GPU tests of rotary positions and of the 4-bit cache,
each of them followed by a read of the device error word, which a failed bounds check
raises."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import pytest  # noqa: E402

from exact_attention_117_b200 import fa  # noqa: E402

FILES = ("test_rotary.py", "test_kv4_cache.py", "test_kv4_attention.py", "test_kv4_precision.py")
# (gigabytes of cache and a long context: nothing that the checks see differently)
LARGE = "not offsets_past_32_bits and not 2_to_the_31 and not long_context"


class AfterEach:
    ran = 0

    @pytest.hookimpl(trylast=True)
    def pytest_runtest_teardown(self, item):
        fa.check_device_error()
        self.ran += 1


def main():
    assert fa.LIB_PATH.endswith("_debug.so"), fa.LIB_PATH
    plugin = AfterEach()
    code = pytest.main([*(os.path.join(HERE, f) for f in FILES), "-m", "gpu", "-k", LARGE, "-x", "-q",
                        "-p", "no:cacheprovider"], plugins=[plugin])
    if code:
        raise SystemExit(int(code))
    fa.check_device_error()
    print(f"debug build: {plugin.ran} cases clean")


if __name__ == "__main__":
    main()
