"""Run tests/test_kvcache_abi.py against another build of libkm_cache.so.

usage: run_with_cache_lib.py <path-to-library> [pytest arguments]
(a child process of test_kvcache_abi.py, which preloads the sanitizer runtime for it)
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, ROOT)

import pytest  # noqa: E402

from means_clustering_amd import kvcache  # noqa: E402

kvcache.LIB_PATH = sys.argv[1]
tests = os.path.join(ROOT, "tests", "test_kvcache_abi.py")
sys.exit(pytest.main([tests, "-q", "-p", "no:cacheprovider", *sys.argv[2:]]))
